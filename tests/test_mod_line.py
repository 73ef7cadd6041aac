"""The line of key tiles that attention with modified scores shares out (CPU).

csrc/kvc_mod_line.cuh is compiled as host code and every CTA's walk is taken: each tile of each unit has to be met once;
a unit that lies in one CTA is finished there and has no piece; and the pieces of the others have to lie in slots of their
own, those that the merge reads, in the order of the CTAs.  Two units in one slot would give one the other's output."""
import math
import os
import shutil
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "paged_kv_cache_kvc_gb300", "csrc", "kvc_mod_line.cuh")

# stdin: lines of heads, CTAs, units, tiles of each unit.  stdout: "s cta segment head unit k0 k1 tiles slot all" and
# "m head unit first ctas slot0", then "e"
PROGRAM = r"""
#include <cstdio>
#include <vector>
#include "%s"
int main() {
    int heads, ctas, units;
    while (scanf("%%d %%d %%d", &heads, &ctas, &units) == 3) {
        std::vector<int32_t> prefix(units + 1, 0);
        for (int u = 0; u < units; ++u) {
            int n;
            if (scanf("%%d", &n) != 1) return 1;
            prefix[u + 1] = prefix[u] + n + kvc::kMtStart;
        }
        for (int c = 0; c < ctas; ++c) {
            kvc::Walk w(prefix.data(), units, heads, c, ctas, false);
            int i = 0;
            for (kvc::Segment s = w.next(); s.ok; s = w.next(), ++i)
                printf("s %%d %%d %%d %%d %%d %%d %%d %%d %%d\n", c, i, s.head, s.unit, s.k0, s.k1, s.tiles, (int)kvc::piece_slot(c, i), (int)s.all());
        }
        const int64_t W = (int64_t)heads * prefix[units], G = ctas < W ? ctas : W;
        for (int h = 0; h < heads; ++h)
            for (int u = 0; u < units; ++u) {
                const int64_t at = (int64_t)h * prefix[units];
                const kvc::Pieces p = kvc::pieces_of(at + prefix[u], at + prefix[u + 1], W, G);
                printf("m %%d %%d %%d %%d %%d\n", h, u, p.first, p.ctas, p.slot0);
            }
        printf("e\n");
    }
    return 0;
}
"""


@pytest.fixture(scope="module")
def walk(tmp_path_factory):
    nvcc = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    nvcc = nvcc if os.path.exists(nvcc) else shutil.which("nvcc")
    if not nvcc:
        pytest.skip("nvcc not available")
    d = tmp_path_factory.mktemp("line")
    (d / "walk.cu").write_text(PROGRAM % HEADER)
    subprocess.check_call([nvcc, "-std=c++17", "-o", str(d / "walk"), str(d / "walk.cu")], cwd=d)

    def run(cases):
        text = "".join(f"{h} {c} {len(t)} {' '.join(map(str, t))}\n" for h, c, t in cases)
        out = subprocess.run([str(d / "walk")], input=text, capture_output=True, text=True, check=True).stdout.split("e\n")
        return [[line.split() for line in x.splitlines()] for x in out[:len(cases)]]
    return run


def hold(heads, ctas, tiles, lines):
    """One case's walk; returns the most segments of a CTA."""
    segments = [tuple(map(int, x[1:])) for x in lines if x[0] == "s"]
    pieces, met, most = {}, {}, 0
    for cta, i, h, u, k0, k1, n, slot, whole in segments:
        assert n == tiles[u] and 0 <= k0 < k1 <= n
        assert k0 == met.get((h, u), 0)          # in the order of the CTAs, no tile twice or left out
        met[h, u] = k1
        most = max(most, i + 1)
        assert whole == (k0 == 0 and k1 == n)
        if not whole:
            assert slot < 2 * ctas
            pieces.setdefault((h, u), []).append((cta, slot))
    assert met == {(h, u): n for h in range(heads) for u, n in enumerate(tiles)}
    used = [s for p in pieces.values() for _, s in p]
    assert len(used) == len(set(used)), "two pieces in one slot"
    for x in lines:
        if x[0] == "m":
            h, u, first, n, slot0 = map(int, x[1:])
            if n == 1:
                assert (h, u) not in pieces
            else:
                assert pieces[h, u] == [(first + t, slot0 if t == 0 else 2 * (first + t)) for t in range(n)]
    return most


def tiles_of(lens):
    return [max(1, -(-(-(-n // 16)) // 4)) for n in lens]   # an empty unit has one tile: it writes its zeros


# lengths of a serving batch: short sequences beside long ones
BATCHES = [[8192] * 32 + [50] * 32, [8192, 50] * 32, [32768] * 8 + [50] * 24, [16384] * 16 + [1] * 16, [32768] * 5 + [16] * 59,
           [64] * 1376, [1 + (7 * i) % 64 for i in range(2048)], [32768] + [500] * 79, [0] * 40 + [5000, 0, 0, 20000], [1], [32768], [20005] * 8]


@pytest.mark.parametrize("heads", [1, 2, 3, 8])
def test_batches(walk, heads):
    cases = [(heads, ctas, tiles_of(b)) for b in BATCHES for ctas in (152, 148, 132)]
    most = [hold(*c, lines) for c, lines in zip(cases, walk(cases))]
    assert max(most) >= 3   # shares that hold whole units between two cut ones are among them


def test_random_lines(walk):
    r = np.random.default_rng(11)
    cases = []
    for _ in range(300):
        units = int(math.exp(r.uniform(0, math.log(400))))
        longest = math.exp(r.uniform(0, math.log(3000)))
        tiles = [max(1, int(math.exp(r.uniform(0, math.log(longest + 1e-9))))) for _ in range(units)]
        cases.append((int(r.integers(1, 9)), int(r.integers(1, 200)), tiles))
    for c, lines in zip(cases, walk(cases)):
        hold(*c, lines)


def test_long_lines_pass_32_bits(walk):
    """Places times CTAs past 2^31, and a line of more than 2^31 places."""
    for case in [(8, 152, [500000] * 40 + [3] * 100), (64, 152, [1 << 24] * 8 + [1])]:
        hold(*case, walk([case])[0])


def test_a_launch_keeps_its_places_inside_32_bits(tmp_path):
    """A call's tables hold up to 2^26 blocks (2^24 tiles a unit), a launch up to 2 048 units a head."""
    nvcc = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    nvcc = nvcc if os.path.exists(nvcc) else shutil.which("nvcc")
    if not nvcc:
        pytest.skip("nvcc not available")
    tiles = sorted({1, 2, 313, 2 ** 19, 2 ** 20, *(2 ** e + d for e in range(2, 25) for d in (-1, 0, 1) if 2 ** e + d <= 2 ** 24)})
    body = "".join(f'printf("%d %d\\n", kvc::units_per_launch({t}), kvc::kMtStart);\n' for t in tiles)
    (tmp_path / "units.cu").write_text(f'#include <cstdio>\n#include "{HEADER}"\nint main() {{\n{body}return 0;\n}}\n')
    subprocess.check_call([nvcc, "-std=c++17", "-o", str(tmp_path / "units"), str(tmp_path / "units.cu")], cwd=tmp_path)
    out = subprocess.check_output([str(tmp_path / "units")], text=True).splitlines()
    for t, line in zip(tiles, out, strict=True):
        units, start = map(int, line.split())
        assert 1 <= units <= 2048 and units * (t + start) < 2 ** 31
        assert units == 2048 or (units + 1) * (t + start) >= 2 ** 31   # no more launches than that takes
