"""The 4-bit route and the rotation where offsets pass 32 bits, and on several
streams and threads at once."""
import threading

import pytest
import torch

import w8a8_int8_quantized_i8_gb300 as i8
from tests import _fp4

pytestmark = pytest.mark.gpu


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_rows_past_four_gigabytes(fmt):
    """2^33 elements: x, its codes and its scales pass 2^32 bytes, 2^32 codes and 2^29 scales."""
    K, rows = 32768, (1 << 18) + 200
    part = torch.randn(256, K, generator=_gen(1), device="cuda").bfloat16()
    x = torch.empty(rows, K, dtype=torch.bfloat16, device="cuda")
    x[:256], x[-256:] = part, part.flip(0)
    x[256:-256] = 0.25
    got = i8.quant_rows_fp4(x, fmt)
    codes, scales, s = _fp4.quantize(part.flip(0).double(), fmt)
    assert torch.equal(got.codes[-256:], codes)
    # the last 256 rows' scales, out of the tiles that hold them
    first = (rows - 256) // 128
    tail = got._replace(codes=got.codes[first * 128:], block_scales=got.block_scales[first:])
    assert torch.equal(_fp4.untile(tail.block_scales, rows - first * 128, K, fmt)[-256:], scales)
    if fmt == "nvfp4":
        assert torch.equal(got.row_scales[-256:].double(), s)
    del x
    w = i8.quant_rows_fp4((torch.randn(64, K, generator=_gen(2), device="cuda") * 0.02).bfloat16(), fmt)
    y = i8.gemm_fp4_bias_bf16(got, w)[-256:].double()
    a = unpacked = _fp4.values(i8.quant_rows_fp4(part.flip(0).contiguous(), fmt))
    b = _fp4.values(w)
    want, size = a @ b.T, a.abs() @ b.abs().T
    assert unpacked.shape == (256, K)
    assert ((y - want).abs() <= 2.0 ** -8 * want.abs() + (K + 4) * 2.0 ** -24 * size).all()
    i8.sync_check()


def test_heads_past_four_gigabytes():
    T, H, D = 300000, 60, 128
    qkv = torch.empty(T, H, D, dtype=torch.bfloat16, device="cuda")
    tail = torch.randn(40, H, D, generator=_gen(3), device="cuda").bfloat16()
    qkv.fill_(0.5)
    qkv[-40:] = tail
    positions = torch.arange(T, dtype=torch.int32, device="cuda")
    inv = (10000.0 ** (-torch.arange(64, device="cuda").double() / 64)).float()
    g = (1 + 0.1 * torch.randn(D, generator=_gen(4), device="cuda")).bfloat16()
    q, k = qkv[:, :50], qkv[:, 50:]
    want = i8.heads_rmsnorm_rotate(tail[:, :50], tail[:, 50:], positions[-40:].contiguous(), inv, g, g)
    i8.heads_rmsnorm_rotate(q, k, positions, inv, g, g, out=(q, k))
    assert torch.equal(q[-40:], want[0]) and torch.equal(k[-40:], want[1])
    i8.sync_check()


def _layers(seed, M, N=768, K=1024):
    g = _gen(seed)
    x = torch.randn(M, K, generator=g, device="cuda").bfloat16()
    return x, *(i8.quant_rows_fp4((torch.randn(N, K, generator=g, device="cuda") * 0.05).bfloat16()) for _ in range(2))


@pytest.mark.parametrize("sizes", [(1, 16), (3, 40), (64, 100), (300, 5), (1000, 1000)])
def test_two_streams_at_once(sizes):
    """CTAs of several calls share SMs, their tensor memory and the clusters' waits with one another."""
    work = [_layers(i, M) for i, M in enumerate(sizes)]
    want = [i8.gated_linear_fp4(x, g, u) for x, g, u in work], [i8.linear_fp4(x, g) for x, g, _ in work]
    streams = [torch.cuda.Stream() for _ in work]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(40):
        for i, (s, (x, g, u)) in enumerate(zip(streams, work)):
            with torch.cuda.stream(s):
                got[i].append((i8.gated_linear_fp4(x, g, u), i8.linear_fp4(x, g)))
    torch.cuda.synchronize()
    i8.sync_check()
    for i in range(2):
        assert all(torch.equal(a, want[0][i]) and torch.equal(b, want[1][i]) for a, b in got[i])


def test_threads_at_once():
    work = [_layers(i, M) for i, M in enumerate((1, 30, 200, 700))]
    want = [i8.gated_linear_fp4(x, g, u) for x, g, u in work]
    torch.cuda.synchronize()
    bad = []

    def run(i):
        x, g, u = work[i]
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(30):
                y = i8.gated_linear_fp4(x, g, u)
            torch.cuda.current_stream().synchronize()
        if not torch.equal(y, want[i]):
            bad.append(i)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(len(work))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    i8.sync_check()
    assert not bad


def test_a_first_call_in_a_capture_and_a_workspace_of_the_caller_s():
    """A width that nothing ran before, quantized and multiplied for the first time while a graph is captured; the
    workspace and the output are the caller's."""
    x, g, u = _layers(9, 45, N=392, K=2080)
    ws = torch.empty(i8.linear_fp4_workspace_bytes(45, g), dtype=torch.uint8, device="cuda")
    y = torch.zeros(45, 392, dtype=torch.bfloat16, device="cuda")
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        i8.linear_fp4(x, g, out=y, workspace=ws)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, i8.linear_fp4(x, g))
    for bad in (ws[:-1], ws[16:]):
        with pytest.raises(i8.I8Error) as e:
            i8.linear_fp4(x, g, out=y, workspace=bad)
        assert e.value.status == 4
    with pytest.raises(ValueError):
        i8.linear_fp4(x, g, workspace=ws.cpu())
    with pytest.raises(TypeError):
        i8.linear_fp4(x, g, workspace=7)


def test_the_output_may_lie_where_the_tokens_do():
    x, g, _ = _layers(11, 70, N=1024, K=1024)
    want = i8.linear_fp4(x, g)
    got = i8.linear_fp4(x, g, out=x)
    assert got is x and torch.equal(x, want)


def test_the_binding_s_refusals_on_the_device():
    x, g, u = _layers(12, 8)
    rows = i8.quant_rows_fp4(x)
    other = i8.quant_rows_fp4(x, "mxfp4")
    wide = i8.quant_rows_fp4(torch.zeros(16, 2048, dtype=torch.bfloat16, device="cuda"))
    bias = torch.zeros(768, device="cuda")
    for call in (lambda: i8.gemm_fp4_bias_bf16(rows, other), lambda: i8.gemm_fp4_bias_bf16(rows, wide),
                 lambda: i8.linear_fp4(x, wide), lambda: i8.linear_fp4(x[:, :1000], g), lambda: i8.linear_fp4(x.t(), g),
                 lambda: i8.gated_linear_fp4(x, g, wide), lambda: i8.gemm_fp4_gated_bf16(rows, g, rows),
                 lambda: i8.linear_fp4(x, g, out=torch.zeros(8, 760, dtype=torch.bfloat16, device="cuda")),
                 lambda: i8.linear_fp4(x, g, torch.zeros(760, dtype=torch.bfloat16, device="cuda")),
                 lambda: i8.quant_rows_fp4(x, out=other), lambda: i8.quant_rows_fp4(x, "mxfp4", out=rows),
                 lambda: i8.quant_rows_fp4(x[0]), lambda: i8.add_rmsnorm_quant_fp4(x, x[:4]),
                 lambda: i8.add_rmsnorm_quant_fp4(x, residual_out=x), lambda: i8.add_rmsnorm_quant_fp4(x, out=other),
                 lambda: i8.gemm_fp4_bias_bf16(rows._replace(codes=rows.codes[:, ::2]), g),
                 lambda: i8.gemm_fp4_bias_bf16(rows._replace(block_scales=rows.block_scales[..., :512]), g),
                 lambda: i8.gemm_fp4_bias_bf16(rows._replace(row_scales=rows.row_scales[:4]), g),
                 lambda: i8.gemm_fp4_bias_bf16(rows._replace(codes=rows.codes.cpu()), g)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: i8.linear_fp4(x.float(), g), lambda: i8.linear_fp4(x, g, bias),
                 lambda: i8.gemm_fp4_bias_bf16(rows._replace(codes=rows.codes.int()), g),
                 lambda: i8.add_rmsnorm_quant_fp4(x, eps="a")):
        with pytest.raises(TypeError):
            call()
    q = torch.zeros(4, 2, 64, dtype=torch.bfloat16, device="cuda")
    p, f = torch.zeros(4, dtype=torch.int32, device="cuda"), torch.ones(32, device="cuda")
    for call in (lambda: i8.heads_rmsnorm_rotate(q, q[:3], p, f), lambda: i8.heads_rmsnorm_rotate(q, q, p[:3], f),
                 lambda: i8.heads_rmsnorm_rotate(q, q, p, f, sections=(16, 16)),
                 lambda: i8.heads_rmsnorm_rotate(q, q, p[None], f), lambda: i8.heads_rmsnorm_rotate(q, q, p, f, f),
                 lambda: i8.heads_rmsnorm_rotate(q, q, p, f, sections=(31,)),
                 lambda: i8.heads_rmsnorm_rotate(q, q, p.expand(5, 4).contiguous(), f, sections=(8, 8, 8, 4, 4)),
                 lambda: i8.heads_rmsnorm_rotate(q, q, p, f, out=(q, q[:2]))):
        with pytest.raises((ValueError, TypeError)):
            call()
    with pytest.raises(i8.I8Error):      # both outputs in one place
        i8.heads_rmsnorm_rotate(q, q, p, f, out=(q, q))
    with pytest.raises(i8.I8Error):      # channels that are no multiple of 8
        i8.linear_fp4(x, i8.quant_rows_fp4(x[:4]))
    i8.sync_check()
