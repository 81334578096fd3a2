// kvc_rope.cu -- append of ragged new tokens to a paged cache with rotary positions (kvc_rope.cuh), with or
// without norms of the heads.
#include <type_traits>

#include "kvc_rope.cuh"

namespace kvc {

template <typename T, int TB, bool VECTOR, bool NORM, bool LATE = false>
__global__ void __launch_bounds__(ROPE_THREADS, 4) append_rope_kernel(const RopeParams p, const __grid_constant__ RopeTable rt) {
    append_rows<T, TB, VECTOR, NORM, LATE>(p, rt, blockIdx.x);
}

// Launch of blocks of tb rows.
static cudaLaunchConfig_t rows_config(cudaLaunchAttribute* attr, int N, int tb, cudaStream_t s) {
    attr->id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr->val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(((unsigned)N + tb - 1) / tb);
    cfg.blockDim = dim3(ROPE_THREADS);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cfg;
}

template <typename T>
static int launch_rope(const RopeParams& p, const RopeTable& t, int sms, cudaStream_t s) {
    // Rows of a block: 4 when that still gives each SM two blocks (the angles' work and the search
    // are shared: 2100 fp32 rows of 24 heads 13.0 us against 15.8 with 1), else 1 (more blocks for
    // a few rows).
    const bool many = p.N >= 8 * sms;
    cudaLaunchAttribute attr[1];
    const cudaLaunchConfig_t cfg = rows_config(attr, p.N, many ? 4 : 1, s);
    const bool vec = t.rot_dim % (2 * Elem<T>::VEC) == 0 && p.D % (2 * Elem<T>::VEC) == 0;
    const bool norm = p.q_norm || p.k_norm;
    auto launch = [&](auto tbs, auto vecs, auto norms) {
        return cudaLaunchKernelEx(&cfg, append_rope_kernel<T, decltype(tbs)::value, decltype(vecs)::value, decltype(norms)::value>,
                                  p, t);
    };
    auto with = [&](auto tbs, auto vecs) { return norm ? launch(tbs, vecs, std::true_type{}) : launch(tbs, vecs, std::false_type{}); };
    using Four = std::integral_constant<int, 4>;
    using One = std::integral_constant<int, 1>;
    const cudaError_t e = many ? (vec ? with(Four{}, std::true_type{}) : with(Four{}, std::false_type{}))
                               : (vec ? with(One{}, std::true_type{}) : with(One{}, std::false_type{}));
    return e != cudaSuccess ? (int)e : (int)cudaGetLastError();
}

int launch_append_rope(int dtype, const RopeParams& p, const RopeTable& t, int sms, cudaStream_t s) {
    return dtype == 0 ? launch_rope<__nv_bfloat16>(p, t, sms, s) : launch_rope<float>(p, t, sms, s);
}

template <typename T>
static int launch_late(const RopeParams& p, const RopeTable& t, cudaStream_t s) {
    cudaLaunchAttribute attr[1];
    const cudaLaunchConfig_t cfg = rows_config(attr, p.N, 4, s);
    const cudaError_t e = p.q_norm ? cudaLaunchKernelEx(&cfg, append_rope_kernel<T, 4, true, true, true>, p, t)
                                   : cudaLaunchKernelEx(&cfg, append_rope_kernel<T, 4, true, false, true>, p, t);
    return e != cudaSuccess ? (int)e : (int)cudaGetLastError();
}
int launch_late_queries(int dtype, const RopeParams& p, const RopeTable& t, cudaStream_t s) {
    return dtype == 0 ? launch_late<__nv_bfloat16>(p, t, s) : launch_late<float>(p, t, s);
}

}  // namespace kvc
