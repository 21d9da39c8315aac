// vts_attend_micro_f16.hip -- the kernels of vts_attend.hpp over microscaled caches, F16.
#include "vts_attend.hpp"

namespace vts {

template <int D, int F>
static hipError_t launch_slots(const AttendParams& p, hipStream_t stream) {
    return p.slots ? launch_mode<F16, D, true, F>(p, stream) : launch_mode<F16, D, false, F>(p, stream);
}

hipError_t launch_attend_micro_f16(int head_dim, int bits, const AttendParams& p, hipStream_t stream) {
    if (bits == 8)
        return head_dim == 64 ? launch_slots<64, 8>(p, stream) : launch_slots<128, 8>(p, stream);
    return head_dim == 64 ? launch_slots<64, 4>(p, stream) : launch_slots<128, 4>(p, stream);
}

}  // namespace vts
