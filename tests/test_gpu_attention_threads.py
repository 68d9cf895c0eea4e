"""fp32 attention called at once by host threads with head sizes that share a
kernel and take different amounts of shared memory: the kernel's limit is the
device's, not the call's.  (The library's entry in tight loops: the interpreter
is let go of during a call.)"""
import threading

import pytest
import torch

import transformer_xl_relative_rel_gb300 as txl
from transformer_xl_relative_rel_gb300 import abi, inputs
from tests.helpers import TOL_F32, device_layer, oracle_full, unit_shape

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from transformer_xl_relative_rel_gb300 import _build
    _build.build()


@pytest.mark.parametrize("sizes", [(8, 20, 32), (33, 48, 64), (65, 96, 128)])
def test_head_sizes_of_one_kernel_at_once(sizes):
    cases = []
    for D in sizes:
        dev, host = device_layer(inputs.unit_layer(unit_shape(1, 2, D, 20, 30), D), torch.float32)
        want = txl.rel_attn_fwd(dev["q"], dev["k"], dev["v"], dev["r"], dev["u"], dev["w"], mem_len=30)
        torch.cuda.synchronize()
        assert abs(want.double().cpu().numpy() - oracle_full(host, 30)).max() <= TOL_F32
        cases.append((D, dev, want))
    entry, failed, start = abi.load_library().txl_rel_attn_fwd, [], threading.Barrier(len(cases))

    def work(D, dev, want):
        try:
            s, out = torch.cuda.Stream(), torch.full_like(want, float("nan"))
            torch.cuda.synchronize()
            args = (*(dev[n].data_ptr() for n in ("q", "k", "v", "r", "u", "w")), 1, 30, 20, 2, D, txl.TXL_F32,
                    out.data_ptr(), s.cuda_stream)
            start.wait()
            states = {entry(*args) for _ in range(4000)}
            s.synchronize()
            failed.extend((D, st) for st in states if st != 0)
            if not torch.equal(out, want):
                failed.append((D, "out"))
        except Exception as e:      # an error of a thread is the test's
            failed.append((D, repr(e)))

    threads = [threading.Thread(target=work, args=c) for c in cases]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed[:5]
    txl.check()
