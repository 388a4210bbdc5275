"""The kernels' shapes of the block norm that no other test compares with the oracle, and its column sums over a
training batch.  Tolerances as in test_gpu_block_norm.py, whose case is used."""
import pytest
import torch

from test_gpu_block_norm import Case, U

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("y_bf16", [False, True])
@pytest.mark.parametrize("h_f32", [False, True])
@pytest.mark.parametrize("d", [528, 768, 896, 1024])
@pytest.mark.parametrize("rows", ["sms", "sms + 1", "4 sms", "4 sms + 1"])
def test_forward_of_a_few_rows_per_sm(lib, rows, d, h_f32, y_bf16):
    """More than a row per SM, at most four: 513 to 1024 columns have a shape of their own."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    T = {"sms": sms, "sms + 1": sms + 1, "4 sms": 4 * sms, "4 sms + 1": 4 * sms + 1}[rows]
    k = d // 16 + T + 2 * h_f32 + y_bf16
    c = Case(T, d, y_bf16=y_bf16, h_f32=h_f32, post=k % 3 != 0, period=[None, 1, 100][k // 2 % 3], seed=d + T)
    c.buffers()
    c.forward(lib)
    lib.sbl_check()
    c.check_forward()


@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("period", [None, 1, 50])
@pytest.mark.parametrize("d", [8208, 16384])
def test_backward_of_light_rows_in_a_pair_of_blocks(lib, d, period, post):
    """At most 13 staged bytes per column beyond 8192 columns: bf16 y and stream, one reader."""
    c = Case(201, d, y_bf16=True, h_f32=False, post=post, period=period, readers=1, seed=d)
    c.buffers()
    c.forward(lib)
    lib.sbl_check()
    c.check_forward()
    c.backward(lib)
    lib.sbl_check()
    c.check_backward()
    c.backward(lib, dH_out=None)  # two bytes per column less
    lib.sbl_check()
    c.check_backward(with_dh=False)


@pytest.mark.parametrize("d", [16, 272, 1040, 4112, 8208])
@pytest.mark.parametrize("readers", [1, 2, 3])
@pytest.mark.parametrize("h_f32", [False, True])
@pytest.mark.parametrize("y_bf16", [False, True])
def test_backward_types_and_readers_apart(lib, y_bf16, h_f32, readers, d):
    """Every pair of types with every number of readers, which decide how many bytes a row stages."""
    c = Case(29, d, y_bf16=y_bf16, h_f32=h_f32, period=8, readers=readers, seed=d + readers)
    c.buffers()
    c.forward(lib)
    lib.sbl_check()
    c.check_forward()
    c.backward(lib)
    lib.sbl_check()
    c.check_backward()


@pytest.mark.parametrize("period", [None, 2048])
def test_column_sums_over_a_training_batch(lib, period):
    """32768 rows against fp64 sums.

    At 2048 columns a lane is 256 threads, two lanes per SM, and each adds its rows in sequence: at most 120 of
    them where the gate rows cut the batch into segments.  On the path of a term: 120 additions, 1 of the pair, 19
    rows of 16 partial rows and 16 of those; and 27 behind the term itself (the mean: 5 in a thread, 5 + 3 in the
    warp and the block; its factors 5, the sum of the readers 2, the products 7).  183 roundings, K = 192.  That
    is 0.7 here, where one row left out changes a column by 1.4 on average."""
    T, d = 32768, 2048
    g = torch.Generator(device="cuda").manual_seed(17)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    bf = torch.bfloat16
    Y, H, dX = rnd(T, d), rnd(T, d).to(bf), [rnd(T, d) for _ in range(3)]
    dH_out = rnd(T, d).to(bf)
    g_pre, g_post = (1 + 0.2 * rnd(d)).to(bf), (1 + 0.2 * rnd(d)).to(bf)
    groups = 1 if period is None else T // period
    gate = None if period is None else rnd(groups, d).to(bf)
    H_out, rstd, dY = torch.empty_like(H), torch.empty(2 * T, device="cuda"), torch.empty_like(H)
    lib.sbl_block_norm(Y, H, g_post, gate, period or 0, 0.75, g_pre, 1e-6, T, d, 0, H_out, None, None, None, rstd)
    got = {k: torch.empty(d, device="cuda") for k in ("dg_pre", "dg_post")}
    got["dgate"] = None if period is None else torch.empty(groups, d, device="cuda")
    n = lib.sbl_block_norm_backward_workspace_bytes(d)
    lib.sbl_block_norm_backward(dX, dH_out, Y, H_out, g_post, gate, period or 0, 0.75, g_pre, rstd, T, d, 0, dY, None,
                                got["dg_post"], got["dg_pre"], got["dgate"], 0,
                                torch.empty(n, dtype=torch.uint8, device="cuda"), n)
    lib.sbl_check()
    zero = lambda *s: torch.zeros(*s, dtype=torch.float64, device="cuda")  # noqa: E731
    want = dict(dg_pre=zero(d), dg_post=zero(d), dgate=zero(groups, d))
    size = dict(dg_pre=zero(d), dg_post=zero(d), dgate=zero(groups, d))
    gp, go = g_pre.double(), g_post.double()
    for i in range(groups):  # in parts: fp64 copies of all of it would not be small
        at = slice(i * T // groups, (i + 1) * T // groups)
        gt = 1.0 if gate is None else gate[i].double()
        r1, r2 = rstd[:T][at].double()[:, None], rstd[T:][at].double()[:, None]
        dxn, mx = sum(x[at].double() for x in dX), sum(x[at].double().abs() for x in dX)
        xh, yh, dh = H_out[at].double() * r2, Y[at].double() * r1, dH_out[at].double()
        t, mt = dxn * gp, mx * gp.abs()
        dh1 = dh + r2 * (t - xh * (t * xh).mean(1, keepdim=True))
        m1 = dh.abs() + r2 * (mt + xh.abs() * (mt * xh.abs()).mean(1, keepdim=True))
        want["dg_pre"] += (dxn * xh).sum(0)
        size["dg_pre"] += (mx * xh.abs()).sum(0)
        want["dg_post"] += (gt * dh1 * yh).sum(0)
        size["dg_post"] += (m1 * yh.abs() * (gt if gate is None else gt.abs())).sum(0)
        want["dgate"][i] = (dh1 * yh * go).sum(0)
        size["dgate"][i] = (m1 * (yh * go).abs()).sum(0)
    for k, v in got.items():
        if v is not None:
            worst = ((v.double() - want[k]).abs() / (192 * U * size[k])).max().item()
            assert worst <= 1.0, (k, worst)
