"""What a prompt's operators refuse before any launch, beyond tests/test_prompt_cpu.py."""
import ctypes

import paged_fp8_kv_gk_gb300 as gk
from test_prompt_cpu import FAKE, no_device, prompt


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
