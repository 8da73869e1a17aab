"""CPU checks of how the package holds its compiled parts."""

import ggml_iq_codebook_amd as iq
from ggml_iq_codebook_amd import layers


def test_library_loads_again_after_the_binding(monkeypatch):
    """The extension module becomes an attribute of the package, `_layers`: no other name
    of the package may be that one."""
    layers._native()
    monkeypatch.setattr(iq, "_lib", None)
    assert iq.load().iq_int8_linear_workspace(40, 8, 70) == 40 * 80 + 160
