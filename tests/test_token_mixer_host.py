"""Host side of the token mixers beside the rule: where their kernels put and find things, at sizes that no test can run.  No GPU
is needed."""
import os
import shutil
import subprocess

import pytest

from gated_delta_rule_gdn_gb300 import build


def compiled(d, text):
    """A program around the headers that the kernels share; its arguments and results are whole numbers."""
    (d / "main.cpp").write_text(text)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(build._nvcc())))
    subprocess.run([shutil.which("g++") or "c++", "-std=c++17", "-fsanitize=undefined", "-fno-sanitize-recover", "-I", os.path.join(cuda, "include"), "-I", build.CSRC, "-I",
                    build.INCLUDE, str(d / "main.cpp"), "-o", str(d / "run")], check=True)
    return lambda *args: [int(v) for v in subprocess.run([str(d / "run"), *map(str, args)], check=True, capture_output=True,
                                                         text=True).stdout.split()]


@pytest.fixture(scope="module")
def places(tmp_path_factory):
    return compiled(tmp_path_factory.mktemp("places"), r'''
#include "paged.h"
#include <cstdio>
#include <cstdlib>
int main(int, char** v) {
    gdn::PagedAttnArgs a{};
    a.c.N = atoi(v[1]); a.Hq = atoi(v[2]); a.splits = atoi(v[3]); a.c.d = atoi(v[4]);
    for (int n = 0; n < a.c.N; ++n)
        for (int h = 0; h < a.Hq; ++h)
            for (int s = 0; s < a.splits; ++s)
                printf("%lld %lld\n", (long long)gdn::paged_attn_tops_at(a, n, h, s), (long long)gdn::paged_attn_sums_at(a, n, h, s));
    printf("%zu\n", gdn::paged_attn_workspace_bytes(a));
}
''')


@pytest.mark.parametrize("N,Hq,splits,d", [(1, 1, 3, 33), (1, 1, 1, 33), (3, 5, 7, 1), (2, 3, 2, 255), (1, 1, 5, 127), (2, 4, 3, 128)])
def test_parts_of_the_attention_in_the_workspace(places, N, Hq, splits, d):
    """Pairs lie on 8 bytes whatever the sizes, and no two pieces overlap."""
    *at, size = places(N, Hq, splits, d)
    if splits == 1:
        assert size == 0
        return
    pairs, sums = at[::2], at[1::2]
    assert all(p % 2 == 0 for p in pairs)
    used = [e for p in pairs for e in range(p, p + 2)] + [e for s in sums for e in range(s, s + d)]
    assert len(set(used)) == len(used) and min(used) == 0 and max(used) + 1 == size // 4 and size % 4 == 0


@pytest.fixture(scope="module")
def parts(tmp_path_factory):
    return compiled(tmp_path_factory.mktemp("parts"), r'''
#include "paged.h"
#include <cstdio>
#include <cstdlib>
int main(int, char** v) {
    const int len = atoi(v[1]), splits = atoi(v[2]), per = gdn::paged_attn_part_tokens(len, splits);
    printf("%d %d", per, gdn::paged_attn_parts(len, per));
    for (int s = 0; s <= splits; ++s) printf(" %d", gdn::paged_attn_part_begin(len, per, s));
}
''')


MOST = 0x7FFFFF00                       # tokens of a sequence that the entry takes


@pytest.mark.parametrize("splits", [1, 2, 3, 7, 304, 1023, 1024])
@pytest.mark.parametrize("length", [0, 1, 127, 128, 129, 8192, 100_003, (1 << 31) - (1 << 21) - 1, (1 << 31) - (1 << 21) + 1, MOST - 1023, MOST - 65536,
                                    MOST - 1, MOST])
def test_parts_of_a_sequence(parts, length, splits):
    """They cover the sequence in order, whatever its length, and are no more than there are places for."""
    per, count, *begin = parts(length, splits)
    assert per >= 128 and per % 64 == 0 and (per == 128 or per - 64 < -(-length // splits))
    assert count <= splits and count == -(-length // per)
    assert begin == [min(length, s * per) for s in range(splits + 1)] and begin[-1] == length


@pytest.fixture(scope="module")
def segments(tmp_path_factory):
    return compiled(tmp_path_factory.mktemp("segments"), r'''
#include "lin.h"
#include <cstdio>
#include <cstdlib>
int main(int, char** v) { printf("%d\n", gdn::lin_segments(atoi(v[1]), atoi(v[2]))); }
''')


@pytest.mark.parametrize("size", [128, 512, 57 * 128, 1 << 20, 1 << 25, 1 << 30])
@pytest.mark.parametrize("length", [0, 1, 127, 128, 129, 4096, (1 << 31) - 65536])
def test_segments_of_a_sequence(segments, length, size):
    assert segments(length, size) == [-(-length // size)]
