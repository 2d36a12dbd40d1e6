"""A stand-in for the compiled library: records the calls that the binding makes, runs no kernel."""
import nvfp4_mixture_experts_gb300 as moe
from nvfp4_mixture_experts_gb300 import build as moe_build

CPU = -1  # what a CPU tensor's get_device() gives
SIZES = ("moe_dispatch_rows_capacity", "moe_mxfp4_scale_bytes", "moe_mxfp4_workspace_size",
         "moe_status_string")  # host arithmetic: the library's own


class StandIn:
    """Has the library's entry points; .calls: (name, arguments) of those that would launch."""

    def __init__(self, lib):
        self.calls = []
        for name in SIZES:
            setattr(self, name, getattr(lib, name))

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            return moe.MOE_OK
        return call


def install(monkeypatch):
    """Puts a stand-in in the library's place, with the CPU as the current device."""
    moe_build.build()
    s = StandIn(moe.load())
    monkeypatch.setattr(moe, "_lib", s)
    monkeypatch.setattr(moe, "_place", lambda stream: (CPU, 0))
    return s
