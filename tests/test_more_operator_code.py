"""Properties of the built device code of the bf16 product and the adapters that
no result shows (CPU: the library's gfx950 code is only read)."""
from __future__ import annotations

import re

from test_operator_code import _kernels


def test_copies_to_lds_go_by_lane_and_own_offsets_alone(tmp_path):
    """A copy to LDS of what is not there has to come back as zeros: its lane's
    offset is behind the buffer's range, whether or not the check counts a
    scalar offset, of which there is none.  Its own offset, whole kilobytes,
    has twelve bits (a larger one would lose its upper bits without an error
    and copy from before the buffer)."""
    kernels = _kernels(tmp_path, "gemm_stream_kernel", "gemm_tiled_kernel", "lora_down_kernel")
    assert {n for k in kernels for n in ("gemm_stream", "gemm_tiled", "lora_down") if n in k} == {
        "gemm_stream", "gemm_tiled", "lora_down"}
    for name, code in kernels.items():
        copies = [i for i in code if i.startswith("buffer_load") and i.split()[-1] == "lds"]
        assert copies, name
        own = set()
        for i in copies:
            m = re.fullmatch(r"buffer_load_dwordx4 v\d+, s\[\d+:\d+\], 0 offen(?: offset:(\d+))? lds", i)
            assert m, (name, i)
            own.add(int(m.group(1) or 0))
        assert own <= ({1024 * i for i in range(4)} if "gemm_tiled" in name else {0}), (name, own)


def test_kernels_spill_no_registers(tmp_path):
    """Nothing of the main loops goes through scratch memory."""
    for name, code in _kernels(tmp_path, "gemm_stream_kernel", "gemm_tiled_kernel", "lora_down_kernel",
                               "lora_up_kernel", "combine_grad_kernel").items():
        assert not [i for i in code if i.startswith("scratch_")], name
