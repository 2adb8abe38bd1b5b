"""The recurrence, append and attention calls of tests/test_checked_cache_gpu.py, run against the bounds-checked library
(SR_LIBRARY=libsr_checked.so): a clean run must end with no SR_DEV_BAD_ACCESS flag and with the definitions' results."""
import os
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
sys.path.insert(0, os.path.dirname(HERE))
sys.path.insert(0, HERE)

import torch  # noqa: E402

import gated_deltanet_state_sr_b200 as sr  # noqa: E402
import test_kv_append_gpu as A  # noqa: E402
import test_linrec_gpu as L  # noqa: E402
import test_paged_attention_gpu as P  # noqa: E402


def flags(ws):
    f = sr.device_status(ws)
    assert f == 0, f"device status 0x{f:x} (0x10: an access outside its buffer)"


if __name__ == "__main__":
    assert sr.CHECKED, "run with SR_LIBRARY=libsr_checked.so"
    ws = sr.workspace(64 << 20)
    for lens, D in (([1, 0, 3], 37), ([63, 1, 0, 7, 300], 64), ([600], 130), ([20, 700], 200)):
        for types in ((L.BF, L.BF), (L.BF, L.F32), (L.F32, L.F32)):
            c = L.make(lens, D, *types, seed=D)
            y, _ = L.check_forward(sr, c, ws=ws)
            flags(ws)
            L.check_backward(sr, c, y, ws=ws)
            flags(ws)
    for new, past, kw in (([5, 0, 40], [3, 20, 0], {}), ([70, 1], [0, 31], dict(d=256, page=128, rot=64, axes=3))):
        A.check(sr, A.make(new, past, seed=1, **kw), ws=ws)
        flags(ws)
    for new, kv, h_q, h_kv, d, page in (([1, 1], [1, 300], 4, 2, 64, 16), ([3, 0, 2], [70, 30, 5000], 8, 2, 128, 64),
                                        ([1], [9000], 4, 1, 256, 32), ([40, 300], [40, 500], 8, 2, 128, 16),
                                        ([130, 5], [131, 3], 4, 1, 256, 128)):
        P.check(sr, P.make(new, kv, h_q, h_kv, d, page, seed=d), ws=ws)
        flags(ws)
    torch.cuda.synchronize()
    print("checked build: every case clean")
