"""The library's table of (device, stream) pairs."""
import ctypes

import pytest

from tests import _gpu

pytestmark = pytest.mark.gpu


def test_sixty_four_streams_with_side_by_side_products():
    """Each of 64 streams may run two products of a backward pass side by side;
    the streams of the library's own take no place in the table.  The 65th pair
    is refused, and emu_shutdown makes room."""
    import torch
    import fp32_emulated_gemm_gb300 as emu
    from tests import _graphs, test_gpu_graphs as t
    rt = _graphs.runtime()
    emu.emu_shutdown()
    case = t.filled(t.LinearBackward(1536, 300, 500, "bf16x9"), 1)
    case.run()
    want = [x.clone() for x in case.outputs]
    torch.cuda.synchronize()
    emu.emu_shutdown()
    handles = [ctypes.c_void_p() for _ in range(65)]
    try:
        for h in handles:
            assert rt.cudaStreamCreateWithFlags(ctypes.byref(h), 1) == 0    # cudaStreamNonBlocking
        for i, h in enumerate(handles):
            stream = torch.cuda.ExternalStream(h.value)
            with torch.cuda.stream(stream):
                if i == 64:
                    with pytest.raises(emu.EmuError) as e:
                        case.run()
                    assert e.value.status == 4
                    break
                for x in case.outputs:
                    x.zero_()
                case.run()
                for x, w in zip(case.outputs, want):
                    assert torch.equal(x, w)
            assert emu.emu_stream_check(stream) == 0
        emu.emu_shutdown()
        with torch.cuda.stream(torch.cuda.ExternalStream(handles[64].value)):
            case.run()
        torch.cuda.synchronize()
    finally:
        torch.cuda.synchronize()
        emu.emu_shutdown()
        for h in handles:
            if h.value:
                rt.cudaStreamDestroy(h)
