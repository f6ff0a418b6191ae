"""CPU replay of the E4M3 GEMM's loads to LDS (csrc/fp8_gemm.hip, fp8_gemm_kernel): for every tile shape, tile,
wavefront, load instruction, lane and chunk -- the repeats past the end, the short last chunk, the slices of K and the
grouped form's gathered rows included -- the bytes that each lane reads lie inside its buffer, the offsets fit the
32 bits that the instruction takes, every LDS destination lies inside its stage, and the fragment reads cover exactly
the stage's rows.  The formulas are written out from the kernel's source; no GPU is involved."""
import numpy as np
import pytest

SHAPES = {"256x256": (256, 256, 2, 4, 2), "256x128": (256, 128, 4, 2, 3), "128x64": (128, 64, 4, 2, 3),
          "256x64": (256, 64, 8, 1, 3)}
CHUNK, AHEAD = 128, 2


def cdiv(a, b):
    return -(-a // b)


def check_tile(shape, m, n, k, nt, mt, n_tiles, m_tiles, slices, rows, x_rows_of, x_total, grouped):
    """rows: rows of X in the tile; x_rows_of(r): row of X relative to the base; x_total: rows from the base on."""
    tn, tm, wn, wm, st = shape
    lw, lx = tn // 64, tm // 64
    kb, nb = cdiv(k, CHUNK), cdiv(n, 128)
    lane = np.arange(64)
    lrow = lane >> 3
    piece = (lane & 7) ^ lrow
    n0 = nt * tn
    ktail = k % CHUNK
    back = np.where((ktail != 0) & (16 * piece >= ktail), 16 * piece - (ktail - 16), 0)
    share_w = 1 if grouped else min(m_tiles, 8)
    share_x = min(32 // share_w, n_tiles)
    lines_w, lines_x = cdiv(tn, share_w), cdiv(tm, share_x)
    assert lines_w + lines_x <= 512
    stage = 128 * tn + 128 * tm + 4 * tm + 4 * 64
    assert st * stage + 4 * 64 <= 160 * 1024 and st * stage >= 2 * tn * tm
    chunks = set()
    for s in range(slices):
        c0, c1 = kb * s // slices, kb * (s + 1) // slices
        assert c0 < c1
        chunks |= {min(c, c1 - 1) for c in range(c0, c1 + st)}
    chunks = np.array(sorted(chunks))

    def inside(off, size, total, per_chunk, sub=None):
        """off [64] from the base, read of `size` bytes at off - sub + chunk * per_chunk; total bytes from the base."""
        for c in (chunks[0], chunks[-1]) if sub is None else chunks:
            o = off - (sub if sub is not None and c == kb - 1 else 0)
            assert o.min() >= 0 and o.max() < 2 ** 32
            a = o.astype(object) + int(c) * per_chunk
            assert min(a) >= 0 and max(a) + size <= total, (m, n, k, nt, mt, c)

    for w in range(8):
        for j in range(lw):
            r = 8 * (w + 8 * j) + lrow
            rn = np.where(n0 + r < n, r, n - 1 - n0)
            inside(rn * k + 16 * piece, 16, (n - n0) * k, CHUNK, back)
            assert 1024 * w + 8192 * j + 1024 <= 128 * tn
        for j in range(lx):
            r = x_rows_of(np.minimum(8 * (w + 8 * j) + lrow, rows - 1))
            inside(r * k + 16 * piece, 16, x_total * k, CHUNK, back)
            assert 1024 * w + 8192 * j + 1024 <= 128 * tm
        if w < lx:
            inside(4 * x_rows_of(np.minimum(64 * w + lane, rows - 1)) * kb, 4, 4 * x_total * kb, 4)
            assert 64 * w + 64 <= tm
        else:
            b0 = n0 // 128
            inside(4 * np.where(b0 + lane < nb, lane, nb - 1 - b0) * kb, 4, 4 * (nb - b0) * kb, 4)
            assert ((n0 & 127) + tn - 1) >> 7 < 64
        # lines brought into L2
        i = 8 * lane + w
        is_w = (i < lines_w) | (i >= lines_w + lines_x)
        rw = np.where(i < lines_w, i, 0) * share_w + mt % share_w
        rw = np.where(n0 + rw < n, rw, n - 1 - n0)
        rx = np.minimum((np.where(is_w, lines_w, i) - lines_w) * share_x + nt % share_x, tm - 1)
        rx = x_rows_of(np.minimum(rx, rows - 1))
        ahead = np.minimum(chunks + AHEAD, kb - 1)
        for c in (ahead[0], ahead[-1]):
            aw, ax = rw * k + CHUNK * c, rx * k + CHUNK * c
            assert aw.min() >= 0 and aw[is_w].max() + 4 <= (n - n0) * k
            assert ax.min() >= 0 and (is_w.all() or ax[~is_w].max() + 4 <= x_total * k)

    # fragment reads: every row of the stage, all of its 8 pieces, by the wavefronts that own it
    l16, g = lane & 15, lane >> 4
    for rows_n, waves, tiles, base in ((tn, wn, tn // wn // 16, 0), (tm, wm, tm // wm // 16, 128 * tn)):
        seen = np.zeros((rows_n, 8), dtype=int)
        for wi in range(waves):
            for t in range(tiles):
                off = base + 128 * l16 + 16 * ((2 * g) ^ (l16 & 7)) + 128 * 16 * wi * tiles + 2048 * t
                for o in (off, off ^ 16):
                    assert (o >= base).all() and (o + 16 <= base + 128 * rows_n).all()
                    np.add.at(seen, ((o - base) // 128, (o - base) % 128 // 16), 1)
        assert (seen == 1).all()


DENSE = [(65, 1, 16), (100, 513, 384), (333, 5000, 17392), (2048, 17408, 5120), (129, 3000, 3088), (257, 300, 4112),
         (700, 259, 16), (64, 17408, 5120)]


@pytest.mark.parametrize("name", list(SHAPES))
@pytest.mark.parametrize("m,n,k", DENSE)
def test_fp8_gemm_sources_in_bounds(name, m, n, k):
    tn, tm = SHAPES[name][:2]
    n_tiles, m_tiles = cdiv(n, tn), cdiv(m, tm)
    for slices in {1, min(8, cdiv(k, CHUNK))}:
        for nt in sorted({0, n_tiles // 2, n_tiles - 1}):
            for mt in sorted({0, m_tiles // 2, m_tiles - 1}):
                check_tile(SHAPES[name], m, n, k, nt, mt, n_tiles, m_tiles, slices, min(m - mt * tm, tm), lambda r: r,
                           m - mt * tm, False)


@pytest.mark.parametrize("t,topk,e,n,k", [(2048, 8, 128, 2048, 4096), (300, 4, 6, 300, 1040), (4200, 8, 4, 16, 128)])
def test_fp8_gemm_grouped_sources_in_bounds(t, topk, e, n, k):
    rng = np.random.default_rng(0)
    pairs = t * topk
    perm = rng.permutation(pairs)
    n_tiles, m_tiles = cdiv(n, 256), cdiv(pairs, 128) + min(e, pairs)
    for first, rows in ((0, 128), (pairs - 1, 1), (pairs // 2, 37)):
        for nt in {0, n_tiles - 1}:
            check_tile(SHAPES["256x128"], pairs, n, k, nt, 0, n_tiles, m_tiles, 1, rows,
                       lambda r: perm[first + r] // topk, t, True)


def test_fp8_gemm_tile_bound_leaves_a_workgroup_for_zero_rows():
    """The m tiles of the grouped launch hold every expert's, and one more if some pair's id is out of range."""
    rng = np.random.default_rng(1)
    for _ in range(2000):
        e = int(rng.integers(1, 12))
        counts = rng.integers(0, 400, size=e) * (rng.random(e) < 0.7)
        invalid = int(rng.integers(0, 3))
        pairs = int(counts.sum()) + invalid
        if pairs:
            used = int(sum(cdiv(int(c), 128) for c in counts))
            assert used + (invalid > 0) <= cdiv(pairs, 128) + min(e, pairs)


def test_fp8_gemm_largest_k_offsets_fit_32_bits():
    k = 1 << 23                     # fp8_gemm_supported
    assert 255 * k + 16 * 7 < 2 ** 32 and 4 * 255 * cdiv(k, CHUNK) < 2 ** 32


@pytest.mark.parametrize("tiles", [1, 7, 8, 60, 61, 160, 544])
def test_gemm_ids_reach_every_tile_once(tiles):
    """The workgroups of a slice: XCD id % 8 takes consecutive tiles, whatever their number."""
    more = tiles & 7
    got = [(i & 7) * (tiles >> 3) + min(i & 7, more) + (i >> 3) for i in range(tiles)]
    assert sorted(got) == list(range(tiles))


@pytest.mark.parametrize("pairs,experts,seed", [(513, 3, 0), (1000, 8, 1), (4096, 128, 2), (600, 1000, 3), (520, 1, 4)])
def test_grouped_places_reach_every_tile_and_zero_row_once(pairs, experts, seed):
    """Every XCD's places: its eighth of the tiles in use, then zero rows, each of them from exactly one place."""
    rng = np.random.default_rng(seed)
    for invalid in (0, 1, pairs // 3, pairs):
        counts = np.bincount(rng.integers(0, experts, pairs - invalid), minlength=experts)
        used = int((-(-counts // 128)).sum())
        per = cdiv(cdiv(pairs, 128) + min(experts, pairs), 8)    # m tiles per XCD
        left, tiles, rows = 8 * per - used, [], []
        for i in range(8 * per):
            xcd, mt = i & 7, i >> 3
            t0, t1 = used * xcd >> 3, used * (xcd + 1) >> 3
            if mt < t1 - t0:
                tiles.append(t0 + mt)
            else:
                assert left > 0
                rows += list(range(pairs - invalid + xcd * per - t0 + mt - (t1 - t0), pairs, left))
        assert sorted(tiles) == list(range(used))
        assert sorted(rows) == list(range(pairs - invalid, pairs))
