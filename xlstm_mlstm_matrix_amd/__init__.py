"""mLSTM cell forward (xLSTM) on AMD MI355X (gfx950).

The compute path is the HIP library ``libmlstm.so`` behind the C ABI in
``include/mlstm.h`` and ``include/mlstm_ops.h``; :mod:`.binding` marshals torch
tensors into it.
"""
from .binding import (BF16, F32, MlstmError, fwd_chunkwise, groupnorm_bwd, groupnorm_fwd,  # noqa: F401
                      lib, linattn_bwd, linattn_fwd, linattn_step, status_string, step, workspace_size)

__version__ = "0.1.0"
