"""GB300 (sm_103a) state-space scans: the Mamba-2 SSD chunked scan, the selective scan with a decay rate per
channel and state, the gated delta rule with the norms of its queries and keys, and what serving them takes (single tokens,
carried windows, 8-bit snapshots).

The compute lives in libssd.so (C ABI, include/ssd.h); this package holds its
thin ctypes binding (``_lib``) and the compiled one of the newer calls (``_binding``), convenience wrappers that allocate outputs and
workspace with torch (``api``), the seeded input generator (``inputs``) and the
build script (``build``).  Importing the package does not load the library; the
first call does, and raises if it has not been built.
"""
from .api import ssd_forward, ssd_backward, Workspace  # noqa: F401
from .api import (selective_scan_forward, selective_scan_backward, SelectiveScanFunction, ssd_step,  # noqa: F401
                  selective_scan_step, conv1d_prompt, conv1d_step, snapshot_store, snapshot_load)
from .api import (gated_delta_forward, gated_delta_backward, GatedDeltaFunction, gated_delta_step, qk_norm_forward,  # noqa: F401
                  qk_norm_backward, QKNormFunction)
