"""Attention over the key/value cache where the blocks' scales, the pages that are seen and the rows' lengths differ
widely inside one call: every row keeps the accuracy of what it sees itself."""
import numpy as np
import pytest
import torch

import context_causal_attention_tcgen05_gb300 as cpa
from gpu_common import _record, check_ok, need_gpu
from oracle import serving
from test_gpu_kv_cache import BF16, F32, Cache, filled, i32, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def reference(c, b, q, L, pos_q, window=0, pos_k=None, k=None, v=None, v_scale=None):
    """out, lse and their bounds for rows q [n, Hq, D] over the first L tokens of sequence b (or over k, v).

    |s| is off by at most D + 8 fp32 roundings of its terms (sabs: the largest sum of their magnitudes) and a weight by
    twice that, the exponential's 2^-21 and, for bf16, its rounding to 11 bits (2^-12); the sum over the keys and the
    division by at most 2^-18; the result is rounded once.  A row's weights are kept in steps of 2^-22 (bf16; fp32 2^-28)
    of its own largest product of a weight and a value scale, half a step off each, and a code is at most 448.  So a score
    is taken relative to a reference that lies up to the spread of the value scales from the row's maximum; the
    difference, at most that spread and 16 in powers of two, is rounded to fp32."""
    bf16 = q.dtype == BF16
    x = q.double().cpu().numpy()
    k = c.values(0, b, L) if k is None else k
    v = c.values(1, b, L) if v is None else v
    pos_k = np.arange(L) if pos_k is None else pos_k
    n, Hq, D = x.shape
    G = Hq // k.shape[1]
    ref, rl, absv, sabs = serving.cache_attention(x, k, v, pos_q, pos_k, True, window)
    if v_scale is None:
        v_scale = c.scales[1][[int(c.table[b][t // c.page]) for t in range(L)]].astype(np.float64)  # [L, Hkv]
    see = pos_k[None] <= pos_q[:, None]
    if window:
        see &= pos_q[:, None] - pos_k[None] < window
    top = np.zeros((n, Hq))
    for h in range(Hq):
        s = np.where(see, (x[:, h] @ k[:, h // G].T) * D**-0.5, -np.inf)
        z = np.where(np.isfinite(rl[h]), rl[h], 0)[:, None]
        top[:, h] = (np.exp(s - z) * v_scale[:, h // G]).max(axis=1, initial=0)
    spread = np.log2(v_scale.max(initial=1e-30) / v_scale.min(initial=1e30)) if L else 0
    ds = (D + 8) * 2.0**-24 * sabs + max(0, spread + 16) * 2.0**-24
    rel = 2 * ds + 2.0**-18 + 2.0**-21 + (2.0**-12 if bf16 else 0)
    bo = ((2.0**-8 if bf16 else 2.0**-24) * np.abs(ref) + rel[:, :, None] * (absv + np.abs(ref)) +
          (see.sum(axis=1)[:, None] * (2.0**-23 if bf16 else 2.0**-29) * 448 * top)[:, :, None] + 1e-44)
    bl = ds.T + 2.0**-19 + 2.0**-22 * np.maximum(np.abs(np.where(np.isfinite(rl), rl, 0)), 1)
    return ref, rl, bo, bl


def check_rows(out, lse, ref, rl, bo, bl, what):
    o, l = out.double().cpu().numpy(), lse.double().cpu().numpy()
    empty = np.isneginf(rl)
    assert np.array_equal(np.isneginf(l), empty), what
    assert np.isfinite(o).all() and (o[empty.T] == 0).all(), what
    worst = [float((np.abs(o - ref) / bo).max()), float((np.abs(np.where(empty, 0, l) - np.where(empty, 0, rl)) / bl).max())]
    _record(f"{what} out", worst[0], 1.0)
    _record(f"{what} lse", worst[1], 1.0)
    assert max(worst) <= 1, (what, worst)


ROWS = [(2, BF16), (4, BF16), (9, BF16), (40, BF16), (140, BF16), (300, BF16), (1, F32), (3, F32), (20, F32)]


@pytest.mark.parametrize("order", ["small first", "large first"])
@pytest.mark.parametrize("what", ["keys", "values", "both"])
@pytest.mark.parametrize("ratio", [2.0**-12, 2.0**-18, 2.0**-33])
@pytest.mark.parametrize("n,dtype", ROWS)
def test_rows_that_see_small_blocks_beside_rows_that_see_large_ones(n, dtype, ratio, what, order):
    """One half of a cache holds keys or values `ratio` times as large as the other's.  Half of the rows see that half
    alone (their queries as much larger, so that their scores matter); the others see large blocks, or both."""
    L, D, page, W = 1300, 64, 16, 600
    half = 656  # whole pages, inside a tile
    c = Cache([L], 2, D, page)
    mag = torch.ones(L, 1, 1, device="cuda")
    small = slice(0, half) if order == "small first" else slice(half, L)
    mag[small] = ratio
    k, v = randn(L, 2, D, dtype=F32), randn(L, 2, D, dtype=F32, seed=1)
    c.append(k * mag if what != "values" else k, v * mag if what != "keys" else v, [L], [0], check=False)
    early = np.arange(n) % 2 == 0
    if order == "small first":  # the first rows see small blocks only, the others both
        pos, window = np.where(early, half - 1 - np.arange(n), L - 1 - np.arange(n)), 0
    else:  # by the window: rows at the end see small blocks only, the others large ones only
        pos, window = np.where(early, L - 1 - np.arange(n) % 40, half - 1 - np.arange(n)), W
    q = randn(n, 4, D, dtype=F32, seed=2)
    if what != "values":
        q[torch.from_numpy(early).cuda()] *= 1 / ratio
    q = q.to(dtype)
    out, lse = cpa.cp_kv_cache_attention(q, *c.args(), i32([L]), i32([0, n]), q_pos=i32(pos), window=window)
    ref = reference(c, 0, q, L, pos, window)
    check_rows(out, lse, *ref, what=f"beside {n} {what} {order}")
    check_ok()


@pytest.mark.parametrize("n,dtype", ROWS)
def test_large_values_under_small_weights(n, dtype):
    """A page whose values are 2^16 as large as the rest, under weights about as small: both halves of the sum count."""
    L, D = 1100, 128
    c = Cache([L], 1, D, 32)
    k, v = randn(L, 1, D, dtype=F32) * 0.2, randn(L, 1, D, dtype=F32, seed=1)
    v[320:352] *= 2.0**16
    k[320:352] -= 8 * np.log(2) / D**0.5  # q is near 1 in every element: 2 * 8 log 2 lower scores
    c.append(k, v, [L], [0], check=False)
    q = (2 + 0.2 * randn(n, 4, D, dtype=F32, seed=2)).to(dtype)
    out, lse = cpa.cp_kv_cache_attention(q, *c.args(), i32([L]), i32([0, n]))
    ref = reference(c, 0, q, L, np.arange(L - n, L))
    check_rows(out, lse, *ref, what=f"small weights {n}")
    check_ok()


@pytest.mark.parametrize("n,dtype,tile", [(1, BF16, 4), (2, BF16, 8), (4, BF16, 16), (70, BF16, 512), (1, F32, 4), (6, F32, 8)])
def test_every_unit_has_its_record(n, dtype, tile):
    """The second launch takes rows and partial results by the records that the first leaves in the workspace, which may
    hold anything before: every row of every head is in one record, and none leads outside the batch or the partial
    results (512 workers' at most)."""
    lens, news = [3000, 0, 40, 700, 2], [n, 2, n, 0, 1]
    c = filled(lens, 2, 128, 32, dtype)
    rows, G = sum(news), 4
    q = randn(rows, 2 * G, 128, dtype=dtype, seed=6)
    ws = torch.full((cpa.cp_workspace_size("kv_attention", rows, 2 * G, 2, 128, cpa._dt(q), len(lens)),), 0x7F,
                    dtype=torch.uint8, device="cuda")
    cu = np.concatenate([[0], np.cumsum(news)])
    out, lse = cpa.cp_kv_cache_attention(q, *c.args(), i32(lens), i32(cu), window=2500, workspace=ws)
    check_ok()
    for b, (m, L) in enumerate(zip(news, lens)):
        r = slice(cu[b], cu[b + 1])
        if m:
            check_rows(out[r], lse[:, r], *reference(c, b, q[r], L, np.arange(L - m, L), 2500), what=f"records {n}")
    slots = rows * G // tile + len(lens)
    records = ws[:slots * 2 * 16].cpu().numpy().view(np.int32).reshape(slots, 2, 4)
    for h in range(2):
        seen = np.zeros(rows * G, int)
        for row, nrows, c0, c1 in records[:, h].tolist():
            assert 0 <= nrows <= tile
            if nrows:
                assert 0 <= row and row + nrows <= rows * G and (c0 == -1 or 0 <= c0 <= c1 < 512)
                seen[row:row + nrows] += 1
        assert (seen == 1).all()


@pytest.mark.parametrize("page", [16, 64, 128])
@pytest.mark.parametrize("n,dtype", [(1, BF16), (5, F32), (70, BF16), (300, BF16)])
def test_pages_that_no_row_sees_need_not_exist(n, dtype, page):
    """Pages before every row's window and behind every row's position may have been given back: their entries are not
    used."""
    L, W, last = 2000, 130, 1500  # the last row's position
    c = filled([L], 2, 128, page, dtype)
    pos = last - n + 1 + np.arange(n)
    lo, hi = (pos[0] - W + 1) // page, last // page + 1
    c.t[4][0, :lo] = -1
    c.t[4][0, hi:] = 10**6
    q = randn(n, 8, 128, dtype=dtype, seed=3)
    out, lse = cpa.cp_kv_cache_attention(q, *c.args(), i32([L]), i32([0, n]), window=W, q_pos=i32(pos))
    check_ok()
    ref = reference(c, 0, q, L, pos, W)
    check_rows(out, lse, *ref, what=f"given back {n} {page}")
    # the window alone: the rows are the last tokens
    c = filled([L], 2, 128, page, dtype)
    c.t[4][0, :(L - n - W + 1) // page] = -1
    out, lse = cpa.cp_kv_cache_attention(q, *c.args(), i32([L]), i32([0, n]), window=W)
    check_ok()
    check_rows(out, lse, *reference(c, 0, q, L, np.arange(L - n, L), W), what=f"given back by window {n} {page}")
    # a page that a row sees is still reported
    c.t[4][0, L // page - 1] = -1
    cpa.cp_kv_cache_attention(q, *c.args(), i32([L]), i32([0, n]), window=W)
    assert cpa.cp_check_device_status() == -9


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("singles,chunk", [(20, 200), (90, 200), (3, 40)])
def test_single_tokens_beside_a_chunk(singles, chunk, dtype):
    """A ragged batch of single tokens and one prompt's chunk, by either kernel."""
    rng = np.random.default_rng(5)
    lens = rng.integers(1, 900, size=singles + 1).tolist()
    news = [1] * (singles + 1)
    lens[singles // 2], news[singles // 2] = 1000, chunk
    c = filled(lens, 2, 128, 64, dtype)
    q = randn(sum(news), 8, 128, dtype=dtype, seed=5)
    cu = np.concatenate([[0], np.cumsum(news)])
    out, lse = cpa.cp_kv_cache_attention(q, *c.args(), i32(lens), i32(cu))
    for b, (n, L) in enumerate(zip(news, lens)):
        r = slice(cu[b], cu[b + 1])
        check_rows(out[r], lse[:, r], *reference(c, b, q[r], L, np.arange(L - n, L)), what=f"beside a chunk {singles}")
    check_ok()


@pytest.mark.parametrize("new,dtype", [(1, F32), (30, F32), (1, BF16), (100, BF16)])
def test_striped_ranks_merge_to_the_whole_they_hold(new, dtype):
    """Each of P ranks caches its striped tokens; their attentions merge into that of the values the ranks hold."""
    P, L, H, Hkv, D = 4, 501, 8, 2, 128
    k, v = randn(L, Hkv, D, dtype=F32), randn(L, Hkv, D, dtype=F32, seed=1)
    q = randn(new, H, D, dtype=dtype, seed=4)
    held = [np.zeros((L, Hkv, D)) for _ in range(2)]
    scale = np.zeros((L, Hkv))
    o = l = None
    for r in range(P):
        n = len(range(r, L, P))
        part = Cache([n], Hkv, D, 32, seed=r)
        part.append(k[r::P].contiguous(), v[r::P].contiguous(), [n], [0], check=False)
        for i in range(2):
            held[i][r::P] = part.values(i, 0, n)
        scale[r::P] = part.scales[1][[int(part.table[0][t // 32]) for t in range(n)]]
        oo, ll = cpa.cp_kv_cache_attention(q, *part.args(), i32([n]), i32([0, new]), q_pos=i32(np.arange(L - new, L)),
                                           k_offset=r, k_stride=P)
        oo = oo.float()
        o, l = (oo, ll) if o is None else cpa.cp_lse_merge(o, l, oo, ll)
    ref, rl, bo, bl = reference(None, 0, q, L, np.arange(L - new, L), pos_k=np.arange(L), k=held[0], v=held[1], v_scale=scale)
    _, _, absv, _ = serving.cache_attention(q.double().cpu().numpy(), *held, np.arange(L - new, L), np.arange(L))
    # each part's result is rounded by itself (its magnitude, weighted, is within absv), its share by its lse's rounding;
    # a merge takes two exponentials, a logarithm, two products, a sum and a quotient
    part = (2.0**-8 if dtype == BF16 else 2.0**-24) * absv
    share = 2 * (bl.T[:, :, None] + 3 * 8 * 2.0**-23) * (absv + np.abs(ref))
    check_rows(o, l, ref, rl, bo + part + share, bl + 3 * 2.0**-21 * np.maximum(1, np.abs(rl)), what=f"striped merge {new}")
    check_ok()


@pytest.mark.parametrize("n,dtype", [(1, BF16), (3, BF16), (16, BF16), (100, BF16), (300, BF16), (1, F32), (2, F32), (40, F32), (150, F32)])
@pytest.mark.parametrize("D", [64, 128])
def test_errors_in_the_2_norm(n, dtype, D):
    """fp32: scores to a few fp32 roundings, weights to 2^-28, so well under 2^-20 of the result (a weight of 13 bits gives
    2^-13).  bf16: the result's rounding, up to 2^-8 of its binade's start and so 2^-8 / sqrt 3 of it in the mean, .736 of
    that for values spread evenly over the binade; weights rounded to 11 bits add under a tenth."""
    lens = [2000, 700]
    c = filled(lens, 2, D, 32, dtype, seed=3)
    q = randn(2 * n, 4, D, dtype=dtype, seed=7)
    out, lse = cpa.cp_kv_cache_attention(q, *c.args(), i32(lens), i32([0, n, 2 * n]))
    bound = 2.0**-20 if dtype == F32 else 1.1 * 0.736 * 2.0**-8 / 3**0.5
    for b in range(2):
        rows = slice(b * n, (b + 1) * n)
        ref, rl, _, _ = reference(c, b, q[rows], lens[b], np.arange(lens[b] - n, lens[b]))
        e = np.linalg.norm(out[rows].double().cpu().numpy() - ref) / np.linalg.norm(ref)
        _record(f"2-norm {n} D={D}", e, bound)
        assert e <= bound
        assert np.abs(lse[:, rows].double().cpu().numpy() - rl).max() <= 2.0**-17 * max(1, np.abs(rl).max())
    check_ok()


@pytest.mark.parametrize("n,dtype", [(1, BF16), (2, BF16), (4, BF16), (40, BF16), (1, F32), (6, F32)])
@pytest.mark.parametrize("D", [64, 128])
def test_a_query_element_that_dwarfs_the_others(n, dtype, D):
    """The first element of every query row is 2^14 times as large as the others, and the keys are zero there: scores are
    made of the others alone."""
    L = 500
    c = Cache([L], 2, D, 32)
    k, v = randn(L, 2, D, dtype=F32), randn(L, 2, D, dtype=F32, seed=1)
    k[..., 0] = 0
    c.append(k, v, [L], [0], check=False)
    q = randn(n, 8, D, dtype=F32, seed=2)
    q[..., 0] = 2.0**14
    q = q.to(dtype)
    out, lse = cpa.cp_kv_cache_attention(q, *c.args(), i32([L]), i32([0, n]))
    ref, rl, bo, bl = reference(c, 0, q, L, np.arange(L - n, L))
    absv = serving.cache_attention(q.double().cpu().numpy(), c.values(0, 0, L), c.values(1, 0, L), np.arange(L - n, L), np.arange(L))[2]
    # elements of q from 2^-17 of the row's largest on are whole, smaller ones within 2^-25 of it (fp32 2^-13, 2^-37)
    x = np.abs(q.double().cpu().numpy())
    lost = (x < (2.0**-17 if dtype == BF16 else 2.0**-13) * 2.0**14) * (2.0**-25 if dtype == BF16 else 2.0**-37) * 2.0**14
    ds = np.stack([(lost[:, h] @ np.abs(c.values(0, 0, L)[:, h // 4]).T).max(axis=1) for h in range(8)], axis=1) * D**-0.5
    check_rows(out, lse, ref, rl, bo + 2 * ds[:, :, None] * (absv + np.abs(ref)), bl + ds.T, what=f"large element {n}")
    check_ok()


@pytest.mark.parametrize("n,dtype", [(3, BF16), (40, BF16), (200, BF16), (300, BF16), (3, F32)])
@pytest.mark.parametrize("where", ["k", "v"])
def test_nan_blocks_and_bad_pages_among_scales_far_apart(where, n, dtype):
    """Keys and values that differ by 2^20 from page to page, a page that does not exist and a NaN block: the tokens of the
    first are hidden, the second reaches the rows that see it alone."""
    L, page = 700, 16
    c = Cache([L], 2, 64, page)
    mag = torch.exp2((torch.arange(L, device="cuda") // page * 7 % 21).float())[:, None, None]
    c.append(randn(L, 2, 64, dtype=F32) / mag, randn(L, 2, 64, dtype=F32, seed=1) * mag, [L], [0], check=False)
    i, late = "kv".index(where), int(c.table[0, 43])  # tokens 688 on, head 1
    c.t[2 + i][late, 1] = float("nan")
    c.t[4][0, 5] = -1
    pos = np.where(np.arange(n) % 2 == 0, 687 - np.arange(n) // 2, 699)
    q = randn(n, 8, 64, dtype=dtype, seed=2)
    out, lse = cpa.cp_kv_cache_attention(q, *c.args(), i32([L]), i32([0, n]), q_pos=i32(pos))
    assert cpa.cp_check_device_status() == -9
    hit = torch.from_numpy(pos >= 688).cuda()
    assert torch.isnan(out[hit][:, 4:]).all() and torch.isnan(lse[4:, hit]).all()
    assert torch.isfinite(out[hit][:, :4]).all() and torch.isfinite(lse[:4, hit]).all()
    keep = np.array([t for t in range(L) if t // page != 5])
    scale = c.scales[1][[int(c.table[0][t // page]) for t in keep]].astype(np.float64)
    ref = reference(c, 0, q, L, pos, pos_k=keep, k=c.values(0, 0, L)[keep], v=c.values(1, 0, L)[keep], v_scale=scale)
    ok = ~hit.cpu().numpy()
    check_rows(out[~hit], lse[:, ~hit], ref[0][ok], ref[1][:, ok], ref[2][ok], ref[3][:, ok], what=f"far apart {n}")
    check_ok()
