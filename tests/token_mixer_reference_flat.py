"""The gradient of a constant decay of linear attention in 64 bits, chunk by chunk with torch, for sequences too long to go token by
token.  test_token_mixer_reference_flat.py checks it against that."""
import torch

CHUNK = 128


def constant_decay(q, k, v, do, g, dhT):
    """q, k, v, do [B, T, H, d] with T a multiple of 128, g [H], dhT [B, H, d, d], no initial state, scale d ** -0.5.

    Returns dg [H] and what it is the sum of, [3, B, H, chunks]: what pairs of tokens have is left out, then with S entering a
    chunk and D leaving it: 128 e^(G_end) <D, S>, sum_i i plus_i (1 for the first token), sum_j (128 - j) minus_j."""
    B, T, H, d = q.shape
    n, scale = T // CHUNK, d ** -0.5
    q, k, v, do = (x.double().transpose(1, 2).unflatten(2, (n, CHUNK)) for x in (q, k, v, do))       # [B, H, n, C, d]
    i = torch.arange(1, CHUNK + 1, device=q.device, dtype=torch.float64)
    G = g.double()[:, None] * i                                                                       # [H, C]
    end, into = torch.exp(G[:, -1:] - G)[..., None], torch.exp(G)[..., None]
    whole = torch.exp(G[:, -1])[:, None, None]
    S = torch.zeros(B, H, d, d, device=q.device, dtype=torch.float64)
    states = []
    for c in range(n):
        states.append(S)
        S = whole * S + (k[:, :, c] * end).transpose(-1, -2) @ v[:, :, c]
    D = dhT.double()
    decay = torch.tril(torch.exp((G[:, :, None] - G[:, None, :]).clamp(max=0)))
    between = torch.clamp(i[:, None] - i[None, :], min=0)            # tokens t with j < t <= i
    parts, pairs = torch.zeros(3, B, H, n, device=q.device, dtype=torch.float64), 0.0
    for c in range(n - 1, -1, -1):
        Q, K, V, O, S = q[:, :, c], k[:, :, c], v[:, :, c], do[:, :, c], states[c]
        plus = scale * into[..., 0] * ((O @ S.transpose(-1, -2)) * Q).sum(-1)
        minus = end[..., 0] * ((V @ D.transpose(-1, -2)) * K).sum(-1)
        parts[0, :, :, c] = CHUNK * whole[:, 0, 0] * (D * S).sum((-1, -2))
        parts[1, :, :, c] = (plus * i).sum(-1)
        parts[2, :, :, c] = (minus * (CHUNK - i)).sum(-1)
        pairs = pairs + (scale * decay * between * (Q @ K.transpose(-1, -2)) * (O @ V.transpose(-1, -2))).sum((0, 2, 3))
        D = whole * D + scale * (Q * into).transpose(-1, -2) @ O
    return parts.sum((0, 1, 3)) + pairs, parts
