"""idx_window_attention_mxfp4 against 64 bits: decode steps, drafted tokens and prompts, windows and sinks, and what
lies in slots that a row does not see."""
import itertools

import pytest
import torch

from _cache_ref import attention, check_attention, starts

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module")
def idx():
    import sparse_attention_indexer_tiles_gb300 as pkg
    pkg.load()
    return pkg


def problem(lens, new, group, heads, D, page, dt, seed=0, behind=0, spare=2):
    g = torch.Generator().manual_seed(seed)
    width = max(-(-max(lens) // page), 1)
    need = [-(-n // page) for n in lens]
    pages = sum(need) + spare
    ids = torch.randperm(pages, generator=g).to(torch.int32)
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
    shape = (pages, heads, page)
    cache = []
    for _ in range(2):
        cache.append(torch.randint(0, 256, (*shape, D // 2), generator=g, dtype=torch.uint8))
        cache.append(torch.randint(122, 127, (*shape, D // 32), generator=g, dtype=torch.uint8))
    T = sum(new) + behind
    q = (1.5 * torch.randn(T, heads * group, D, generator=g)).to(TYPES[dt])
    return dict(q=q, cache=cache, table=table, lens=torch.tensor(lens, dtype=torch.int32), q_start=starts(new))


def call(idx, p, **kw):
    dev = "cuda"
    stats = idx.Stats()
    uniform = kw.pop("uniform", False)
    got = idx.idx_window_attention_mxfp4(p["q"].to(dev), *(c.to(dev) for c in p["cache"]), p["table"].to(dev),
                                         p["lens"].to(dev), q_start=None if uniform else p["q_start"].to(dev),
                                         stats=stats, **kw)
    torch.cuda.synchronize()
    return [x.cpu() for x in got], stats.read()["status"]


def check(idx, p, window=0, sink=0, status=0, **kw):
    got, st = call(idx, p, window=window, sink=sink, **kw)
    assert st == status
    ref = attention(p["q"], p["cache"], p["table"], p["lens"], p["q_start"], window, sink, kw.get("scale"))
    check_attention(got, ref, p["q"].dtype, int(p["lens"].max()), p["q"].shape[2])
    outside = ~ref[5]
    assert (got[0][outside] == 0).all() and (got[1][outside] == 0).all()
    return got


@pytest.mark.parametrize("D,page,dt", list(itertools.product([64, 128], [16, 32, 64, 128], ["bf16", "fp16"])))
def test_decode(idx, D, page, dt):
    check(idx, problem([1, 40, 333], [1, 1, 1], 4, 2, D, page, dt), uniform=True)


@pytest.mark.parametrize("group", [1, 2, 5, 7, 8, 9, 16, 33])
def test_groups(idx, group):
    check(idx, problem([70, 129], [1, 1], group, 2, 128, 64, "bf16", seed=group))


@pytest.mark.parametrize("lens", [[1], [15], [16], [17], [31], [32], [33], [63], [64], [65], [127, 128, 129], [513], [2000]])
def test_lengths(idx, lens):
    check(idx, problem(lens, [1] * len(lens), 3, 1, 64, 32, "fp16", seed=lens[0]))


@pytest.mark.parametrize("window,sink", [(1, 0), (1, 1), (16, 4), (31, 0), (32, 5), (33, 33), (100, 0), (100, 17), (100, 64),
                                         (400, 4), (5000, 4)])
def test_windows_of_single_tokens(idx, window, sink):
    check(idx, problem([600, 3, 90, 205], [1, 1, 1, 1], 4, 2, 128, 16, "bf16", seed=window), window, sink)


@pytest.mark.parametrize("window,sink", [(0, 0), (1, 0), (3, 2), (20, 4), (64, 1), (200, 40)])
@pytest.mark.parametrize("group,dt", [(1, "bf16"), (3, "fp16"), (8, "bf16")])
def test_several_tokens(idx, window, sink, group, dt):
    check(idx, problem([7, 130, 250, 64], [7, 2, 16, 5], group, 2, 64, 32, dt, seed=window), window, sink)


@pytest.mark.parametrize("window,sink", [(0, 0), (50, 3), (130, 0)])
@pytest.mark.parametrize("D,dt", [(64, "fp16"), (128, "bf16"), (128, "fp16")])
def test_prompts(idx, window, sink, D, dt):
    check(idx, problem([300, 210, 17], [300, 130, 17], 4, 1, D, 64, dt, seed=D, behind=3), window, sink)


def test_requests_without_tokens_and_tokens_behind_the_last(idx):
    p = problem([50, 60, 0, 70], [3, 0, 0, 4], 2, 2, 128, 16, "bf16", behind=5)
    out = torch.full((12, 4, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((12, 4), 7.0, device="cuda")
    got, st = call(idx, p, window=20, sink=2, out=out, lse=lse, max_q=4)
    assert st == 0 and (got[0][7:] == 7).all() and (got[1][7:] == 7).all()
    check_attention(got, attention(p["q"], p["cache"], p["table"], p["lens"], p["q_start"], 20, 2), torch.bfloat16, 70, 128)


@pytest.mark.parametrize("path", [-1, 1])
def test_rows_that_see_nothing(idx, path):
    """More new tokens than slots: the first ones have no position."""
    p = problem([2, 0], [5, 3], 3, 1, 64, 16, "fp16")
    check(idx, p, options={"row_split": path})
    check(idx, p, window=2, sink=1, options={"row_split": path})


@pytest.mark.parametrize("path", [-1, 1])
def test_rows_that_see_nothing_do_not_look_at_q(idx, path):
    p = problem([2, 50], [6, 4], 3, 1, 64, 16, "bf16", seed=3)
    p["q"][:4] = torch.tensor([float("nan"), float("inf"), -float("inf"), float("nan")])[:, None, None].bfloat16()
    check(idx, p, options={"row_split": path})
    check(idx, p, window=9, options={"row_split": path})


@pytest.mark.parametrize("T", [1, 300])
def test_a_table_without_pages(idx, T):
    """No slot can be cached: every row sees nothing, whatever the path would be, and no cache is needed."""
    z = lambda *s: torch.zeros(*s, dtype=torch.uint8, device="cuda")  # noqa: E731
    lens, table = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros(1, 0, dtype=torch.int32, device="cuda")
    q = torch.randn(T, 64, 128, device="cuda").bfloat16()
    for pages in (0, 3):
        for path in (0, 1):
            out, lse = idx.idx_window_attention_mxfp4(q, z(pages, 8, 16, 64), z(pages, 8, 16, 4), z(pages, 8, 16, 64),
                                                      z(pages, 8, 16, 4), table, lens, options={"row_split": path})
            assert (out == 0).all() and (lse == -float("inf")).all()


def test_scales_that_fp16_does_not_hold_on_the_dense_path(idx):
    """A scale of 2^14 and more counts as a NaN scale there; 2^13 is held."""
    p = problem([120], [60], 4, 1, 64, 16, "fp16", seed=13)
    page = int(p["table"][0, 5])
    p["cache"][3][page, 0, 4, 1] = 127 + 13
    check(idx, p, 30, 2, options=DENSE)
    p["cache"][3][page, 0, 4, 1] = 127 + 14
    q = dict(p, cache=[c.clone() for c in p["cache"]])
    q["cache"][3][page, 0, 4, 1] = 255
    got, _ = call(idx, p, window=30, sink=2, options=DENSE)
    check_attention(got, attention(q["q"], q["cache"], q["table"], q["lens"], q["q_start"], 30, 2), torch.float16, 120, 64)
    check(idx, p, 30, 2, options={"row_split": -1})


def test_long_rows_take_splits(idx):
    p = problem([9000, 100], [1, 1], 2, 1, 64, 128, "bf16", seed=3)
    check(idx, p)
    check(idx, p, window=6000, sink=9)
    check(idx, problem([5000], [4], 8, 1, 128, 64, "fp16", seed=4))


@pytest.mark.parametrize("where", ["k", "v"])
@pytest.mark.parametrize("new", [1, 6])
def test_nan_scales_reach_only_rows_that_see_them(idx, where, new):
    p = problem([100, 100, 100], [new] * 3, 4, 2, 128, 16, "bf16", seed=new)
    sf = p["cache"][1 if where == "k" else 3]
    for b, slot in ((0, 50), (1, 98), (2, 0)):
        sf[int(p["table"][b, slot // 16]), 1, slot % 16, 2] = 255
    for row in p["table"]:                       # slots past the last one hold anything
        sf[int(row[100 // 16]), :, 100 % 16:] = 255
    check(idx, p)
    check(idx, p, window=20, sink=0)
    check(idx, p, window=20, sink=1)


@pytest.mark.parametrize("path", [-1, 1])
@pytest.mark.parametrize("D,dt", [(64, "fp16"), (128, "bf16")])
@pytest.mark.parametrize("new,window,sink", [(1, 37, 0), (1, 37, 5), (1, 1, 0), (1, 0, 0), (3, 20, 33), (7, 70, 1)])
def test_what_no_row_sees_changes_no_bit(idx, new, window, sink, D, dt, path):
    lens = [1, 31, 33, 100, 257]
    p = problem(lens, [min(n, new) for n in lens], 4, 2, D, 16, dt, seed=window + sink)
    options = {"row_split": path}
    want = check(idx, p, window, sink, options=options)
    g = torch.Generator().manual_seed(new)
    seen = torch.zeros(p["cache"][0].shape[0], 16, dtype=torch.bool)
    for b, n in enumerate(lens):
        for j in range(n):
            if window == 0 or j < sink or j > n - min(n, new) - window:
                seen[int(p["table"][b, j // 16]), j % 16] = True
    wild = torch.tensor([0, 1, 90, 254, 255], dtype=torch.uint8)
    for x in p["cache"]:
        is_sf = x.shape[-1] == D // 32
        other = wild[torch.randint(0, 5, x.shape, generator=g)] if is_sf else 255 - x
        x.copy_(torch.where(seen[:, None, :, None], x, other))
    got, st = call(idx, p, window=window, sink=sink, options=options)
    assert st == 0 and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_a_later_token_with_huge_values_leaves_the_ones_before(idx):
    p = problem([64], [8], 2, 1, 128, 16, "bf16", seed=11)
    page = int(p["table"][0, 3])
    p["cache"][3][page, 0, 12:] = 250            # V of the last four tokens: 2^123 times codes
    check(idx, p, window=40)
    p["cache"][1][page, 0, 14:] = 200            # and K: its logits leave nothing to the others
    got, _ = call(idx, p, window=40)
    ref = attention(p["q"], p["cache"], p["table"], p["lens"], p["q_start"], 40)
    o, lse = got[0].double(), got[1].double()
    assert torch.isfinite(o[:6]).all() and ((o[:4] - ref[0][:4]).abs() <= 2.0 ** -6 * ref[2][:4] + 1e-3).all()
    assert ((lse[:6] - ref[1][:6]).abs() <= 1e-3).all()


@pytest.mark.parametrize("spread", [20, 26, 27, 30, 60, 100])
def test_scales_of_v_that_lie_far_apart(idx, spread):
    p = problem([70, 33], [1, 1], 4, 1, 128, 32, "bf16", seed=spread)
    g = torch.Generator().manual_seed(spread)
    sf = p["cache"][3]
    sf[torch.rand(sf.shape, generator=g) < 0.3] = 126 - spread
    sf[torch.rand(sf.shape, generator=g) < 0.1] = 0
    check(idx, p)


def test_pages_outside_the_window_need_not_exist(idx):
    p = problem([640, 200], [2, 1], 4, 2, 64, 16, "fp16", seed=5)
    window, sink = 50, 4
    full = check(idx, p, window, sink)
    for b, n in enumerate([640, 200]):
        first = (n - 2 - window) // 16           # at least the oldest page of the window
        p["table"][b, 1:first] = torch.tensor([-1, -7, 1 << 30, 2 ** 31 - 1] * 20)[:first - 1]
    got, st = call(idx, p, window=window, sink=sink)
    assert st == 0 and torch.equal(got[0], full[0]) and torch.equal(got[1], full[1])


def test_bad_arguments_on_the_device_are_reported(idx):
    p = problem([100, 50], [1, 1], 2, 1, 64, 16, "bf16")
    p["table"][0, 2] = 1000
    assert call(idx, p)[1] == 2
    for lens in ([-1, 50], [113, 50]):
        p = problem([100, 50], [1, 1], 2, 1, 64, 16, "bf16")
        p["lens"] = torch.tensor(lens, dtype=torch.int32)
        got, st = call(idx, p)
        assert st == 2
        ref = attention(p["q"], p["cache"], p["table"], torch.tensor([0, 50]), p["q_start"])
        assert torch.allclose(got[0][1].double(), ref[0][1], atol=2e-2)
    for start in ([0, 2, 1], [-1, 1, 2], [0, 1, 9]):
        p = problem([100, 50], [1, 1], 2, 1, 64, 16, "bf16")
        p["q_start"] = torch.tensor(start, dtype=torch.int32)
        assert call(idx, p)[1] == 2
    p = problem([100, 50], [3, 1], 2, 1, 64, 16, "bf16")
    assert call(idx, p, max_q=2)[1] == 2


def test_queries_of_any_size_and_rows_that_are_not_finite(idx):
    for dt, scales in (("bf16", [1e-30, 1.0, 1e30, 0.0]), ("fp16", [1e-4, 1.0, 100.0, 0.0])):
        p = problem([90] * 4, [1] * 4, 3, 2, 128, 32, dt, seed=1)
        s = torch.tensor(scales)[:, None, None]
        p["q"] = (p["q"].float() * s).to(TYPES[dt])
        for scale in (None, 1e-3, -0.1):
            if dt == "bf16":
                p["q"][2] = (p["q"][2].float() * 1e-30).to(TYPES[dt]) if scale is None else p["q"][2]
            check(idx, p, scale=scale)
    p = problem([90] * 3, [1] * 3, 3, 2, 128, 32, "bf16", seed=1)
    p["q"][1, 2, 5] = float("nan")
    p["q"][1, 4, 5] = float("inf")
    got, _ = call(idx, p)
    rows = torch.isnan(got[1])
    assert rows[1, 2] and rows[1, 4] and rows.sum() == 2
    assert torch.isnan(got[0][1, 2]).all() and torch.isfinite(got[0][0]).all() and torch.isfinite(got[0][1, 3]).all()


def test_slices_of_a_projection(idx):
    p = problem([100, 50, 77], [2, 1, 3], 4, 2, 64, 16, "bf16", seed=2)
    full = check(idx, p)
    wide = torch.zeros(6, 8 * 64 + 264, dtype=torch.bfloat16)
    wide[:, 8:8 + 512] = p["q"].flatten(1)
    p["q"] = wide.to("cuda")[:, 8:8 + 512].unflatten(1, (8, 64))
    got, st = call(idx, p)
    assert st == 0 and torch.equal(got[0], full[0]) and torch.equal(got[1], full[1])


def test_the_bound_on_the_new_tokens_does_not_matter(idx):
    p = problem([300, 20], [30, 1], 4, 2, 128, 64, "bf16", seed=8)
    for max_q in (30, 31, 0):
        for max_len in (300, 0):
            check(idx, p, 64, 4, max_q=max_q, max_len=max_len)


DENSE = {"row_split": 1}


def test_a_wait_that_runs_out_is_reported(idx):
    """Only the dense path waits for copies."""
    made = idx.idx_window_attention_mxfp4_plan(1, 600, 600, 64, 8, 64, 640, 0, 0)
    assert made["dense"] and made["splits"] == 1     # every part has a second tile
    got, st = call(idx, problem([600], [600], 8, 8, 64, 64, "bf16"), options={"test_stall_us": 2000})
    assert st & 1
    check(idx, problem([300], [64], 8, 1, 64, 64, "bf16"), options=DENSE)


@pytest.mark.parametrize("D,dt,window,sink", list(itertools.product([64, 128], ["bf16", "fp16"], [0, 1, 100], [0, 3, 90])))
def test_the_dense_path(idx, D, dt, window, sink):
    """Ragged requests, an odd and an even number of row tiles, tiles at the end of a page."""
    p = problem([330, 61, 100], [130, 61, 70], 6, 2, D, 16, dt, seed=D + window, behind=2)
    check(idx, p, window, sink, max_q=130, max_len=330, options=DENSE)


@pytest.mark.parametrize("group", [1, 3, 40, 64, 128])
def test_groups_on_the_dense_path(idx, group):
    new = [200 if group == 1 else 70]
    p = problem([600], new, group, 1, 64, 32, "bf16", seed=group)
    check(idx, p, 64, 5, options=DENSE)


def test_splits_of_the_dense_path(idx):
    made = idx.idx_window_attention_mxfp4_plan(1, 20, 20, 16, 1, 128, 20000, 0, 0)
    assert made["dense"] and made["splits"] > 1
    check(idx, problem([20000], [20], 16, 1, 128, 64, "bf16", seed=6))
    p = problem([6000], [20], 8, 1, 128, 64, "bf16", seed=6)
    check(idx, p, options=DENSE)
    check(idx, p, 2500, 100, options=DENSE)


@pytest.mark.parametrize("where", ["k", "v"])
def test_nan_scales_on_the_dense_path(idx, where):
    p = problem([200, 150], [70, 90], 4, 2, 128, 16, "bf16", seed=4)
    sf = p["cache"][1 if where == "k" else 3]
    for b, slot in ((0, 150), (1, 149), (0, 3)):
        sf[int(p["table"][b, slot // 16]), 1, slot % 16, 2] = 255
    sf[int(p["table"][0, 12]), :, 8:] = 255      # past the last slot
    check(idx, p, 30, 0, options=DENSE)
    check(idx, p, 30, 4, options=DENSE)


@pytest.mark.parametrize("dt,spread", [("bf16", 10), ("bf16", 40), ("fp16", 8)])
def test_large_scales_on_the_dense_path(idx, dt, spread):
    """Scales up to 2^(spread + 4): bf16 takes two products above 2^15."""
    p = problem([200], [90], 4, 1, 128, 16, dt, seed=spread)
    g = torch.Generator().manual_seed(spread)
    sf = p["cache"][3]
    sf[torch.rand(sf.shape, generator=g) < 0.3] = 127 + spread
    p["cache"][1][:] -= 5
    check(idx, p, options=DENSE)


def test_a_prompt_in_chunks(idx):
    """The same rows whether a prompt comes at once or in chunks: each chunk attends to what is in the cache."""
    p = problem([400], [400], 4, 2, 64, 32, "fp16", seed=9)
    whole = check(idx, p, 90, 7)
    for lo, hi, path in ((0, 100, 1), (100, 101, 0), (101, 390, 1), (390, 400, -1)):
        part = dict(p, q=p["q"][lo:hi].contiguous(), lens=torch.tensor([hi], dtype=torch.int32), q_start=starts([hi - lo]))
        got = check(idx, part, 90, 7, max_len=400, options={"row_split": path})
        err = (got[0].float() - whole[0][lo:hi].float()).abs().max()
        assert err <= 2e-2
