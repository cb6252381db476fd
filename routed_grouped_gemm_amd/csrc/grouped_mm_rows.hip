// The plain products of the weight-streaming kernel (grouped_mm_rows.h), the
// joining of a product split along K, and their launches.
#include <algorithm>

#include "grouped_mm_rows.h"

namespace {

// The sum of a split product's parts, in their order, rounded once: 4 values
// per lane, for the rows that belong to a group.
__global__ __launch_bounds__(256)
void mm_join_kernel(MmP p) {
    int lo, hi, end;
    group_rows(p, 0, lo, hi);
    group_rows(p, p.G - 1, hi, end);
    const int n4 = p.N / 4;
    const int64_t total = (int64_t)p.R_max * n4, stride = (int64_t)gridDim.x * 256;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += stride) {
        const int row = (int)(i / n4), a = (int)(i - (int64_t)row * n4) * 4;
        if (row < lo || row >= end) continue;
        const float* src = p.partial + (size_t)row * p.N + a;
        f32x4 v = *(const f32x4*)src;
        for (int s = 1; s < p.parts; ++s) {
            const f32x4 e = *(const f32x4*)(src + (size_t)s * p.R_max * p.N);
            v = f32x4{v[0] + e[0], v[1] + e[1], v[2] + e[2], v[3] + e[3]};
        }
        *(u32x2_t*)((uint16_t*)p.out + (size_t)row * p.out_ld + a) =
            u32x2_t{pack16(v[0], v[1], p.out_f16), pack16(v[2], v[3], p.out_f16)};
    }
}

template <int EL, int MODE>
int launch_few(const MmP& p, int rows, hipStream_t stream) {
    const int e = rows > 32 ? launch_rows<EL, MODE, 4>(p, stream) : launch_rows<EL, MODE, 2>(p, stream);
    if (e || p.parts == 1) return e;
    const int64_t lanes = (int64_t)p.R_max * (p.N / 4);
    mm_join_kernel<<<(int)std::min<int64_t>((lanes + 255) / 256, 4 * device_cu_count()), 256, 0, stream>>>(p);
    return (int)hipGetLastError();
}

}  // namespace

int moe_launch_mm_rows(const void* params, int el, int kind, int rows, hipStream_t stream) {
    const MmP& p = *(const MmP*)params;
    if (el == kElFp8) return launch_few<kElFp8, kMmNK>(p, rows, stream);
    if (el == kElF16) return kind ? launch_few<kElF16, kMmKN>(p, rows, stream) : launch_few<kElF16, kMmNK>(p, rows, stream);
    return kind ? launch_few<kElBf16, kMmKN>(p, rows, stream) : launch_few<kElBf16, kMmNK>(p, rows, stream);
}
