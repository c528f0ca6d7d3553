"""An adapter backward call without rows that wants gx alone: nothing to do, and no refusal."""
import ctypes

from test_lora_host import ERR_ARG, _backward


def test_empty_gx_alone_is_no_argument_error(e4b):
    """The empty gx of the binding has a NULL pointer; without a GPU the call ends at the device check."""
    none = dict(gx=None, ga=None, gb=None)
    assert e4b._c_lora_bwd(ctypes.byref(_backward(e4b, S=0, gx_base=None, g=None, x=None, z=None, **none)), None) != ERR_ARG
    assert e4b._c_lora_bwd(ctypes.byref(_backward(e4b, S=1, **none)), None) == ERR_ARG
