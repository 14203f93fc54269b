"""What a prompt's operators refuse before any launch, beyond tests/test_prompt_cpu.py."""
import ctypes

import pytest

import paged_fp8_kv_gk_gb300 as gk
from test_prompt_cpu import FAKE, no_device, prompt, shape


@no_device
def test_timeout_hook_arguments():
    L, p, bits = gk.lib(), ctypes.c_void_p(FAKE), ctypes.c_uint32(5)
    pr = prompt()
    # prompt, plan, bytes, q, stride, k, stride, v, stride, sinks, out, out_f32, tries, stream, bits
    args = [ctypes.byref(pr), p, gk.gk_prompt_plan_bytes(pr), p, 4096, p, 512, p, 512, None, p, None, 5, None,
            ctypes.byref(bits)]
    for i, v, want in ((12, 0, 1), (12, -3, 1), (12, (1 << 18) + 1, 1), (14, None, 1), (0, None, 1), (1, None, 3), (3, None, 1),
                       (10, None, 1), (0, ctypes.byref(prompt(head_dim=128)), 2)):
        a = list(args)
        a[i] = v
        assert L.gk_selftest_prompt_attn_timeout(*a) == want, i


@no_device
def test_outputs_that_overlap_inputs():
    """Refused however little they share; neighbours, and outputs between the rows of an input, are not
    (they get as far as the missing device)."""
    L, G = gk.lib(), gk.GK_ERR_CUDA
    T, Hq, H = 5, 16, 2
    pr = prompt(num_seqs=1, num_q_heads=Hq, num_kv_heads=H, q_tokens=T, k_tokens=T)
    plan, at = 1 << 30, 1 << 24
    n = gk.gk_prompt_plan_bytes(pr)
    row, stride = Hq * 128, 2 * 65536            # q's bytes; rows far apart

    def call(q=at, k=at + (1 << 22), v=at + (2 << 22), out=at + (3 << 22), f32=at + (4 << 22), sinks=None, plan=plan,
             pr=pr, q_stride=stride // 2, kv_stride=4096):
        return L.gk_prompt_attn(ctypes.byref(pr), plan, n, q, q_stride, k, kv_stride, v, kv_stride, sinks, out, f32, None)
    assert call() == G and call(f32=None) == G
    size = T * row                               # out's bytes; f32 has twice as many
    for t in range(T):
        q_row = at + t * stride
        for out, want in ((q_row, 1), (q_row + row, G), (q_row + row - 16, 1), (q_row - size, G), (q_row - size + 16, 1),
                          (q_row + 2 * row, G)):
            assert call(out=out, f32=None) == want, (t, out - q_row)
            assert call(f32=out, out=at + (5 << 22)) == (1 if q_row - 2 * size < out < q_row + row else G), (t, out - q_row)
    assert call(out=at + (T - 1) * stride + row) == G and call(out=at + T * stride) == G
    for name, first in (("k", at + (1 << 22)), ("v", at + (2 << 22))):
        for t in (0, T - 1):
            r = first + t * 8192
            assert call(out=r, f32=None) == 1 and call(out=r + H * 128, f32=None) == (1 if t < T - 1 else G), name
            assert call(out=r + H * 128 - 16, f32=None) == 1
        assert call(out=first - size, f32=None) == G
    assert call(sinks=at + (3 << 22) + size - 4) == 1 and call(sinks=at + (3 << 22) + size) == G
    assert call(out=plan) == 1 and call(out=plan + n - 256) == 1 and call(out=plan + n) == G
    assert call(f32=at + (3 << 22) + size - 16) == 1 and call(f32=at + (3 << 22) + size) == G
    # one token: its stride says nothing
    one = prompt(num_seqs=1, num_q_heads=Hq, num_kv_heads=H, q_tokens=1, k_tokens=1)
    n1 = gk.gk_prompt_plan_bytes(one)
    assert n1 <= n
    assert call(pr=one, q_stride=0, out=at, f32=None) == 1
    assert call(pr=one, q_stride=0, kv_stride=0, out=at + row, f32=None) == G


def test_most_items():
    """The kernel's place in a plan, (item, kv head), runs up to two grids past the last in 32 bits: what comes
    nearer to them than 2^16 is refused."""
    def size(q):
        return gk.gk_prompt_plan_bytes(prompt(num_seqs=1, num_q_heads=128 * 8, q_tokens=q))
    most = (2 ** 31 - 1 - 2 ** 16) // 8           # a token a tile
    assert size(most) > 32 * most and size(most + 1) == 0 and size(2 ** 28 - 1) == 0
    with pytest.raises(gk.GkError):
        gk.new_prompt_plan(prompt(num_seqs=1, num_q_heads=128 * 8, q_tokens=most + 1))


@no_device
def test_linear_factors_without_an_inverse():
    L, p = gk.lib(), ctypes.c_void_p(FAKE)
    for factor, want in ((5e-324, 1), (5e-309, 1), (6e-309, gk.GK_ERR_CUDA), (1e-300, gk.GK_ERR_CUDA), (1e300, gk.GK_ERR_CUDA)):
        params = gk.RopeParams.make(64, 1e4, scaling="linear", factor=factor)
        assert L.gk_rope_table(ctypes.byref(params), 3, p, p, p, None) == want, factor


@no_device
def test_misaligned_slots_and_scales():
    """A pointer to int32 or fp32 that is no multiple of four: refused, not left to the GPU."""
    L, p = gk.lib(), ctypes.c_void_p(FAKE)
    arr = (ctypes.c_void_p * 2)(FAKE, FAKE)
    kv = gk.KvCacheC(k_bufs=ctypes.cast(arr, ctypes.c_void_p), v_bufs=ctypes.cast(arr, ctypes.c_void_p))
    # layer0, n_layers, n_tokens, k, v, strides, cos, sin, k_scale, v_scale, slots, active, kv, stream
    write = [0, 4, 10, p, p, 1280, 128, p, p, p, p, p, p, p, ctypes.byref(kv), None]
    read = [0, 4, 10, ctypes.byref(kv), p, p, p, p, p, p, p, None]
    for call, args, where in ((L.gk_kv_write, write, (9, 10, 11, 12)), (L.gk_kv_read, read, (4, 5, 6, 7))):
        assert call(ctypes.byref(shape()), *args) == gk.GK_ERR_CUDA
        for i in where:
            for off in (1, 2, 3):
                a = list(args)
                a[i] = ctypes.c_void_p(FAKE + off)
                assert call(ctypes.byref(shape()), *a) == 1, (i, off)


class Buffer:
    """What a KvCache asks of a buffer when it is made, and no more."""
    is_cuda = True

    def __init__(self, *shape):
        self.shape = shape

    def dim(self):
        return len(self.shape)

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return FAKE


def test_a_cache_is_made_of_what_it_needs():
    """Buffers are asked for their sizes and device by the calls that check them, not when the cache is
    made (which took a quarter longer so, and refused buffers that the decode calls take)."""
    k, v = Buffer(9, 2, 16, 64, 2), Buffer(9, 2, 32, 64)
    kv = gk.KvCache([k, k], [v, v])
    assert kv.k_layout == gk.GK_K_PACKED and kv.c.k_bufs
    kv = gk.kv_stacked(Buffer(2, 9, 2, 32, 64), Buffer(2, 9, 2, 32, 64))
    assert kv.k_layout == gk.GK_K_PLAIN
    assert gk.KvCache([FAKE], [FAKE], k_layout=gk.GK_K_PLAIN).held() == (None, None)
