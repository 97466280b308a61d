"""Launches of the calls that move rows by index and of the adjusting of logits, on the CPU.

A process that loads a recorder in front of the HIP runtime makes calls with addresses that nothing
reads: each launch is written down instead of made.  No GPU takes part, so sizes go up to the
documented limits, which no card's memory holds."""
import json
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

RECORDER = r"""
#include <stddef.h>
typedef struct { unsigned x, y, z; } dim3;
static dim3 g, b;
static size_t shared;
static void *at;
static unsigned launches[4096][4];
static int held;
unsigned __hipPushCallConfiguration(dim3 grid, dim3 block, size_t lds, void *stream) {
    g = grid; b = block; shared = lds; at = stream;
    return 0;
}
unsigned __hipPopCallConfiguration(dim3 *grid, dim3 *block, size_t *lds, void **stream) {
    *grid = g; *block = b; *lds = shared; *stream = at;
    return 0;
}
unsigned hipLaunchKernel(const void *f, dim3 grid, dim3 block, void **args, size_t lds, void *stream) {
    (void)f; (void)args; (void)lds; (void)stream;
    if (held < 4096) {
        launches[held][0] = grid.x; launches[held][1] = grid.y; launches[held][2] = grid.z;
        launches[held][3] = block.x * block.y * block.z;
        ++held;
    }
    return 0;
}
unsigned hipGetLastError(void) { return 0; }
int recorded(unsigned *to) {
    int n = held;
    for (int i = 0; i < n * 4; ++i) to[i] = launches[i / 4][i % 4];
    held = 0;
    return n;
}
"""

CALLER = r"""
import ctypes, json, sys
recorder = ctypes.CDLL(sys.argv[2], mode=ctypes.RTLD_GLOBAL)
sys.path.insert(0, sys.argv[1])
import sorting_lsd_radix_amd as rs
held = (ctypes.c_uint * (4 * 4096))()
out = []
for name, args in json.loads(sys.stdin.read()):
    getattr(rs, name)(*args, stream=0)
    n = recorder.recorded(held)
    out.append([list(held[4 * i:4 * i + 4]) for i in range(n)])
print(json.dumps(out))
"""


@pytest.fixture(scope="module")
def launches_of(tmp_path_factory):
    folder = tmp_path_factory.mktemp("recorder")
    source, library = str(folder / "recorder.c"), str(folder / "recorder.so")
    with open(source, "w") as f:
        f.write(RECORDER)
    subprocess.run(["gcc", "-O1", "-shared", "-fPIC", "-o", library, source], check=True)

    def of(*calls):
        """[[grid x, y, z, threads of a block], ...] for each (name, arguments)."""
        r = subprocess.run([sys.executable, "-c", CALLER, ROOT, library], input=json.dumps(calls), text=True,
                           capture_output=True, timeout=120)
        assert r.returncode == 0, r.stdout + r.stderr
        return json.loads(r.stdout.strip().splitlines()[-1])
    return of


# addresses 2^42 apart, which nothing reads
A, B, C, D, E, F = (i << 42 for i in range(1, 7))
ELEM = {0: 4, 1: 2, 2: 2}
TEMP = (1 << 41, 1 << 40)   # address and size


def embed_grad(n, vocab, width, et=2, tt=2, gap=0, accumulate=0):
    return ["rs_embed_tokens_grad", [et, A, width, B, n, vocab, width, 1.0, accumulate, tt, C, width + gap, *TEMP]]


def fits(launches):
    for x, y, z, threads in launches:
        assert 0 < x and x * threads < 1 << 32, (x, threads)   # work items of a grid dimension
        assert 0 < y <= 65535 and z == 1, (y, z)
        assert x * y < 1 << 32, (x, y)                         # blocks, which kernels count in 32 bits
        assert threads != 256 or x * y * 4 <= 1 << 32, (x, y)  # and the waves of these


# tokens, rows, width, element type, table's type, elements between rows: tables from 64 GB to the largest
LARGE = [
    (3, 600, 1 << 26, 2, 2, 0), (1, 5, 1 << 27, 0, 0, 0), (3, 600, 1 << 25, 2, 0, 0), (5000, 1 << 20, 1 << 17, 1, 1, 0),
    (20000, 1 << 18, 1 << 20, 2, 2, 0), (1000, 1 << 29, 512, 0, 0, 0), (7, (1 << 30) - 1, 256, 2, 2, 0),
    (7, (1 << 30) - 1, 256, 2, 0, 3), (1, 1000, 1 << 28, 2, 2, 0), (100, 1 << 27, 2048, 0, 0, 1),
]


@pytest.mark.parametrize("case", LARGE)
def test_tables_filled_beside_the_sort(launches_of, case):
    """Every launch fits a grid; the launches before the sums have a lane for each 16 bytes of a table
    without gaps, and the sums' none: they write rows, and zeros beside them would race."""
    n, vocab, width, et, tt, gap = case
    launches, = launches_of(embed_grad(n, vocab, width, et, tt, gap))
    fits(launches)
    sort = [l for l in launches if l[3] == 1024 and l is not launches[-1]]
    sums = [l for l in launches if l[3] == 256]
    assert len(sums) == 1
    if gap == 0:
        assert sum(x * y * threads for x, y, _, threads in sort) * 16 >= vocab * width * ELEM[tt]
    chunks = -(-width * ELEM[et] // 1024)   # of 64 vectors; a wave for each and a piece of 8 tokens or more
    blocks = -(-(-(-n // 8)) * chunks // 4)
    x, y, _, _ = sums[0]
    assert x * y <= max(blocks, 65536) + 65536 * (blocks > 65536), (x, y)


@pytest.mark.parametrize("et", [0, 1, 2])
def test_largest_calls_fit_a_grid(launches_of, et):
    """Matrices of 2^38 elements, by rows and by width, and as many rows as there may be."""
    top = (1 << 30) - 1
    calls = []
    for rows, width in ((top, 256), (1 << 27, 2048), (1 << 20, 1 << 18), (256, (1 << 30) - 1)):
        ids, few = min(rows, top // 2), min(1000, (1 << 38) // width)
        calls += [
            ["rs_gather_choices", [et, A, width, B, rows, C, D, rows, 1, width, E, width]],
            ["rs_gather_choices", [et, A, width, B, rows, C, None, 1, 1, width, E, width]],
            ["rs_gather_choices_grad", [et, A, width, rows, B, width, C, D, rows, 1, width, E, width, F]],
            ["rs_combine_choices", [et, A, width, rows, B, C, rows, 1, width, D, width]],
            ["rs_combine_choices_grad", [et, A, width, B, width, C, rows, D, E, rows, 1, width, F, width, 7 << 42]],
            ["rs_embed_tokens", [et, A, width, B, rows, rows, width, 2.0, C, width]],
            ["rs_adjust_logits", [et, A, width, rows, width, None, 0, 0, None, None, None, None, None, None, 0, None, 0, 0,
                                  None, 0, et, B, width]],
            embed_grad(0, rows, width, et, et), embed_grad(ids, few, width, et, 0),
            embed_grad(ids, few, width, et, 0, accumulate=1),
        ]
    for (name, args), launches in zip(calls, launches_of(*calls)):
        assert launches, (name, args)
        fits(launches)
