"""How the microscaled operators are called: streams, memory, devices."""
import numpy as np
import pytest
import torch

from test_gpu_mx import fill, mx, random_bits  # noqa: F401  (mx is the module's fixture)

pytestmark = pytest.mark.gpu

BUSY = 60_000_000      # cycles that keep a stream occupied: some 30 ms


def calls(mx):
    """Calls that allocate their result, [2000, 1024] BF16, each with its value on the
    current stream."""
    rng = np.random.default_rng(2)
    a, _ = fill(mx, "e4m3", random_bits(rng, 2000, 1024, 0.5))
    w, _ = fill(mx, "e4m3", random_bits(rng, 1024, 1024, 0.5))
    gate, up = mx.dequantize(a), mx.dequantize(a)
    g8, u8 = mx.MxTensor.empty("e4m3", 2000, 1024), mx.MxTensor.empty("e4m3", 2000, 1024)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    fns = {"dequantize": lambda s: mx.dequantize(a, stream=s), "matmul": lambda s: mx.matmul(a, w, status=status, stream=s),
           "swiglu": lambda s: mx.swiglu(gate, up, g8, u8, stream=s)}
    return {n: (f, f(None)) for n, f in fns.items()}


@pytest.mark.parametrize("name", ["dequantize", "matmul", "swiglu"])
@pytest.mark.parametrize("as_int", [False, True])
def test_result_is_memory_of_its_stream(mx, name, as_int):
    call, want = calls(mx)[name]
    side = torch.cuda.Stream()
    stream = side.cuda_stream if as_int else side
    torch.cuda.synchronize()
    # a block that the current stream has given back but still works on
    x = torch.full_like(want, 7.0)
    y = torch.zeros_like(want)
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)
    y.copy_(x)
    at = x.data_ptr()
    del x
    out = call(stream)
    assert out.data_ptr() != at
    torch.cuda.synchronize()
    assert bool((y == 7.0).all()) and torch.equal(out, want)
    # a result that is dropped while its stream has yet to write it
    with torch.cuda.stream(side):
        torch.cuda._sleep(BUSY)
    out = call(stream)
    at = out.data_ptr()
    del out
    x = torch.full_like(want, 5.0)
    assert x.data_ptr() != at
    torch.cuda.synchronize()
    assert bool((x == 5.0).all())


def test_forms_whose_memory_was_released_and_taken_again(mx):
    """As a gathered tensor's is between steps: the calls use the memory that a form
    has now, and refuse one that has none."""
    from lossless_bf16_exponent_codec_gb300 import binding as B
    R, C = 700, 900
    bits = random_bits(np.random.default_rng(5), R, C)
    t, value = fill(mx, "e4m3", bits)
    x = mx.dequantize(t)
    store = t.codes.untyped_storage()
    n, at = store.nbytes(), t.codes.data_ptr()
    torch.cuda.synchronize()
    store.resize_(0)
    with pytest.raises(B.EzError):
        mx.dequantize(t)
    taken = [torch.full((n,), 17, dtype=torch.uint8, device="cuda") for _ in range(4)]
    store.resize_(n)
    assert t.codes.data_ptr() != at
    mx.quantize(x, row=t)
    assert torch.equal(mx.dequantize(t), x)         # 8-bit values are their own rounding
    assert all(bool((k == 17).all()) for k in taken)


def test_status_word_of_a_device(mx):
    """One word to a device, however it is spelt: the one that products without a
    word of their own report to."""
    from lossless_bf16_exponent_codec_gb300 import binding as B
    word = mx.status_word("cuda")
    n = torch.cuda.current_device()
    for device in (f"cuda:{n}", torch.device("cuda"), torch.device("cuda", n)):
        assert mx.status_word(device) is word
    a, _ = fill(mx, "e4m3", random_bits(np.random.default_rng(1), 4, 64))
    good = mx.matmul(a, a)
    assert int(word.item()) == 0
    try:
        B.ez_mx_wait_limit(0)
        mx.matmul(a, a)
    finally:
        B.ez_mx_wait_limit()
    assert int(word.item()) == 8
    word.zero_()
    assert torch.equal(mx.matmul(a, a), good) and int(word.item()) == 0
    with pytest.raises(ValueError, match="CUDA device"):
        mx.status_word("cpu")
