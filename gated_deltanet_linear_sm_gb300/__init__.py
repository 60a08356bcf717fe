"""GB300-native Gated DeltaNet speculative / MTP decode step, and the calls
around it.

The compute is the sm_103a CUDA kernels in libgdnspec (C ABI, include/gdnspec.h);
this package holds its Python binding, its build step and the seeded
synthetic-input generator.
"""
from .binding import (BF16, F16, F32, GdnError, LibraryMissing, gdn_dims, gdn_prefill,  # noqa: F401
                      gdn_prefill_chunked, gdn_spec_decode, gdn_spec_decode_conv, library_path, load_library, prepare, status_str, version)
from .ops import (PreparedOp, gdn_conv_prefill, gdn_ssm_decode, gdn_ssm_dims, gdn_ssm_prefill,  # noqa: F401
                  gdn_step_tables, gdn_tables_dims, gdn_verify_dims, gdn_verify_drafts, prepare_conv_prefill,
                  prepare_ssm_decode, prepare_ssm_prefill, prepare_step_tables, prepare_verify_drafts,
                  ssm_prefill_workspace)
