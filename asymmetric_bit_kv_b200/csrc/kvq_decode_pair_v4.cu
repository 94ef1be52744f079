// decode_pair_kernel instances with 4-bit values (1, 2 or 4 value groups per head).
#include "kvq_decode_pair.cuh"

namespace kvq {
namespace tc {

cudaError_t launch_pair_v4(int ngrp, const DecodeParams& p, const MmaPlan& mp, const WindowTables* win,
                           cudaStream_t stream) {
  if (ngrp == 1) return launch_pair_instance<4, 1>(p, mp, win, stream);
  if (ngrp == 2) return launch_pair_instance<4, 2>(p, mp, win, stream);
  if (ngrp == 4) return launch_pair_instance<4, 4>(p, mp, win, stream);
  return cudaErrorInvalidValue;
}

const void* fn_pair_v4(int ngrp, bool win) {
  if (ngrp == 1) return pair_instance_fn<4, 1>(win);
  if (ngrp == 2) return pair_instance_fn<4, 2>(win);
  if (ngrp == 4) return pair_instance_fn<4, 4>(win);
  return nullptr;
}

}  // namespace tc
}  // namespace kvq
