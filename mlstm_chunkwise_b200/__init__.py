"""B200-native (sm_100a) chunkwise mLSTM behind a C ABI: forward, backward and
the single-token step; the gated delta rule (the sibling cell with delta-rule
writes) in the same forms; and the layer norm of the cells' output.

The computation runs in ``libmlstm_fw.so`` (hand-written CUDA kernels; see
``include/mlstm_fw.h``).  This package only builds that library
(``build.py``), marshals arguments into it (``api.py``) and draws seeded
synthetic inputs (``inputs.py``).
"""
from .api import (MlstmError, gated_delta_bw, gated_delta_chunkwise,  # noqa: F401
                  gated_delta_bw_saved, gated_delta_fw, gated_delta_fw_train, gated_delta_step,
                  gated_delta_train_sizes, gated_delta_workspace_size, head_norm,
                  head_norm_bw, head_norm_fw, substep_workspace_size, last_device_error, mlstm_bw,
                  mlstm_bw_saved, mlstm_chunkwise, mlstm_fw, mlstm_fw_chunk_states,
                  mlstm_fw_parallel, mlstm_fw_train, mlstm_step, set_watchdog, train_sizes,
                  workspace_size)
