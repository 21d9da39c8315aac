// vts_attend.hip -- the kernels of vts_attend.hpp over 16-bit caches.
#include "vts_attend.hpp"

namespace vts {

hipError_t launch_attend(int dtype, int head_dim, const AttendParams& p, hipStream_t stream) {
    if (dtype == BF16) {
        if (head_dim == 64)
            return p.slots ? launch_mode<BF16, 64, true, 16>(p, stream)
                           : launch_mode<BF16, 64, false, 16>(p, stream);
        return p.slots ? launch_mode<BF16, 128, true, 16>(p, stream)
                       : launch_mode<BF16, 128, false, 16>(p, stream);
    }
    if (head_dim == 64)
        return p.slots ? launch_mode<F16, 64, true, 16>(p, stream)
                       : launch_mode<F16, 64, false, 16>(p, stream);
    return p.slots ? launch_mode<F16, 128, true, 16>(p, stream)
                   : launch_mode<F16, 128, false, 16>(p, stream);
}

}  // namespace vts
