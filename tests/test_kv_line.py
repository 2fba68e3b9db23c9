"""The token attention kernel's line of work (csrc/kv_line.h), compiled here for the CPU and
compared with a model in Python's whole numbers."""
import ctypes
import random
import subprocess
from pathlib import Path

import pytest

CSRC = Path(__file__).resolve().parents[1] / "nvfp4_block_scaled_04_gb300" / "csrc"
TILE, EXTRA = 64, 3

SOURCE = """
#include "kv_line.h"
using namespace nvfp4;
namespace {
template <int ROWS>
int pieces(const ArLine& a, const ArSeq* s, unsigned ctas, unsigned cta, uint64_t* pre, uint64_t* per_out, ArItem* out, int room) {
  pre[0] = 0;
  for (int b = 0; b < a.batch; ++b) pre[b + 1] = pre[b] + ar_seq_units<64, ROWS, 3>(a, s[b]);
  ArPiece<64, ROWS, 3> piece(a, pre[a.batch], ctas, cta);
  *per_out = piece.per;
  int n = 0;
  auto seq = [&](int b) { return s[b]; };
  while (n < room && piece.next(a, pre, seq, out[n])) ++n;
  return n;
}
}  // namespace
extern "C" void partly(int p0, int p1, int window, int sinks, int j0, int tile, int* out) {
  const KvPartly x = kv_partly(p0, p1, window, sinks);
  out[0] = x.a0, out[1] = x.a1, out[2] = x.b0, out[3] = x.b1, out[4] = x.meets(j0, tile);
}
extern "C" int line_pieces(int rows, const ArLine* a, const ArSeq* s, unsigned ctas, unsigned cta, uint64_t* pre, uint64_t* per,
                           ArItem* out, int room) {
  switch (rows) {
    case 8: return pieces<8>(*a, s, ctas, cta, pre, per, out, room);
    case 16: return pieces<16>(*a, s, ctas, cta, pre, per, out, room);
    case 24: return pieces<24>(*a, s, ctas, cta, pre, per, out, room);
    default: return pieces<32>(*a, s, ctas, cta, pre, per, out, room);
  }
}
"""


class Line(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("batch", "heads", "group", "window", "sinks")] + [("cap", ctypes.c_int64)]


class Seq(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("row0", "n", "len")]


class Item(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("done", "h", "r0", "n_rows", "row0", "p0", "p1", "key_end", "st", "w0", "count",
                                            "i0", "i1", "b")] + [(n, ctypes.c_uint) for n in ("first_cta", "last_cta")]


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    d = tmp_path_factory.mktemp("line")
    (d / "line.cpp").write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-Wall", "-Werror", f"-I{CSRC}", str(d / "line.cpp"), "-o",
                    str(d / "line.so")], check=True)
    return ctypes.CDLL(str(d / "line.so"))


class Cut:
    def __init__(self, lib, rows, line, seqs, ctas):
        self.lib, self.rows, self.line, self.ctas = lib, rows, line, ctas
        self.seqs = (Seq * len(seqs))(*seqs)
        self.pre = (ctypes.c_uint64 * (len(seqs) + 1))()
        self.per = ctypes.c_uint64()

    def __call__(self, cta, room=4096):
        out = (Item * room)()
        n = self.lib.line_pieces(self.rows, ctypes.byref(self.line), self.seqs, self.ctas, cta, self.pre, ctypes.byref(self.per),
                                 out, room)
        return out[:n]


@pytest.mark.parametrize("rows", [8, 16, 24, 32])
@pytest.mark.parametrize("seed", range(12))
def test_every_tile_is_somebodys_once(lib, rows, seed):
    g = random.Random(1000 * rows + seed)
    batch, heads, group = g.choice((1, 2, 9, 60)), g.choice((1, 2, 8)), g.choice((1, 3, 4, 8, 40))
    window = g.choice((0, 0, 1, 50, 700))
    line = Line(batch, heads, group, window, g.choice((0, 3, 200)) if window else 0, g.choice((1 << 20, 1024)))
    seqs, row0 = [], 0
    for _ in range(batch):
        n = g.choice((0, 1, 1, 2, 5, 40))
        seqs.append(Seq(row0, n, g.choice((0, 1, n, 64, 300, 5000))))
        row0 += n
    ctas = g.choice((1, 7, 152, 304))
    cut = Cut(lib, rows, line, seqs, ctas)
    seen = {}
    for cta in range(ctas):
        for it in cut(cta):
            s = seqs[it.b]
            assert it.row0 == s.row0 and 0 <= it.h < heads and it.r0 % rows == 0
            assert it.n_rows == min(rows, s.n * group - it.r0) > 0
            assert it.p0 == s.len - s.n + it.r0 // group and it.p1 == s.len - s.n + (it.r0 + it.n_rows - 1) // group
            assert it.key_end == min(s.len, line.cap)
            assert 0 <= it.i0 <= it.i1 <= it.count and it.first_cta <= cta <= it.last_cta
            parts = seen.setdefault((it.b, it.h, it.r0), [])
            parts.append((cta, it.i0, it.i1, it.count, it.first_cta, it.last_cta))
    assert set(seen) == {(b, h, r) for b, s in enumerate(seqs) for h in range(heads) for r in range(0, s.n * group, rows)}
    for parts in seen.values():
        # one after another, from the first tile to the last, in the CTAs that the item names
        count = parts[0][3]
        assert [p[0] for p in parts] == list(range(parts[0][4], parts[0][5] + 1))
        assert parts[0][1] == 0 and parts[-1][2] == count
        assert all(a[2] == b[1] for a, b in zip(parts, parts[1:]))


@pytest.mark.parametrize("rows,group,heads,news,length", [
    (8, 8, 8, [131072, 131072], 131072),         # 2^32 and a little more
    (8, 4, 8, [1, 400000, 3], 1 << 20),
    (32, 128, 4, [300000, 300000], 300000),
])
def test_lines_longer_than_32_bits(lib, rows, group, heads, news, length):
    line = Line(len(news), heads, group, 0, 0, 1 << 24)
    seqs, row0 = [], 0
    for n in news:
        seqs.append(Seq(row0, n, length))
        row0 += n
    ctas = 304
    cut = Cut(lib, rows, line, seqs, ctas)
    per_item = -(-length // TILE) + EXTRA
    blocks = [-(-n * group // rows) for n in news]
    ends = [0]
    for x in blocks:
        ends.append(ends[-1] + x * heads * per_item)
    assert ends[-1] > 1 << 32
    per = -(-ends[-1] // ctas)
    for cta in (0, 1, 77, 150, 151, 152, 302, 303):
        items = cut(cta, 64)
        assert list(cut.pre) == ends and cut.per.value == per
        u, end = cta * per, min((cta + 1) * per, ends[-1])
        for it in items:
            # the model: the next item on the line whose tiles (not what follows them) lie at or past u
            while True:
                b = max(x for x in range(len(news)) if ends[x] <= u)
                item, i0 = divmod(u - ends[b], per_item)
                rb, h = divmod(item, heads)
                n = news[b]
                p1 = length - n + (min((rb + 1) * rows, n * group) - 1) // group
                count = p1 // TILE + 1
                start = u - i0
                i1 = min(end - start, per_item)
                u = start + i1
                if i0 < count:
                    break
            assert (it.b, it.h, it.r0, it.i0, it.i1, it.count) == (b, h, rb * rows, i0, min(i1, count), count)
            assert (it.first_cta, it.last_cta) == (start // per, (start + count - 1) // per)
        assert items


@pytest.mark.parametrize("window", [0, 1, 2, 3, 7, 20])
@pytest.mark.parametrize("sinks", [0, 1, 5, 40])
def test_positions_that_some_rows_see_and_others_do_not(lib, window, sinks):
    """Against every row's mask; a tile has some exactly where one of its positions is such (a tile that is looked at
    without need costs a wait: a single row has none at all)."""
    out = (ctypes.c_int * 5)()
    for p0 in range(-3, 30):
        for p1 in range(p0, p0 + 9):
            def sees(p, j):
                return j <= p and (not window or p - j < window or j < sinks)
            want = [j for j in range(0, 45) if len({sees(p, j) for p in range(p0, p1 + 1)}) == 2]
            for j0 in range(0, 44, 4):
                lib.partly(p0, p1, window, sinks, j0, 4, out)
                a0, a1, b0, b1, meets = out
                got = [j for j in range(0, 45) if a0 <= j < a1 or b0 <= j < b1]
                assert got == want
                assert max(0, a1 - a0) <= p1 - p0 and max(0, b1 - b0) <= p1 - p0
                assert bool(meets) == any(j0 <= j < j0 + 4 for j in want), (p0, p1, j0)
