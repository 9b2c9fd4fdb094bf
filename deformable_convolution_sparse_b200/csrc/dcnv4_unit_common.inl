// Host-side helpers of the translation units that hold one operator family
// each (dcnv4_mx.cu, dcnv4_predictor_backward.cu, dcnv4_orthogonalize.cu).
// Included inside their anonymous namespace, after dcnv4_host_common.inl.

// Launches with programmatic stream serialisation (DCNV4_PDL=0: plain): every
// thread of `kern` executes griddepcontrol.wait before its first global access.
// The one exception is pred_grad_w_kernel, which waits at its end: the launch
// directly before it has to be pred_grad_y_kernel, which writes nothing that it
// touches, and whose CTAs let it start only after a wait of their own.
template <typename... KA, typename... A>
int launch_chained(void (*kern)(KA...), dim3 grid, int threads, size_t smem, cudaStream_t stream, const A&... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    const char* pe = std::getenv("DCNV4_PDL");
    cfg.numAttrs = (pe && *pe == '0') ? 0 : 1;
    if (cudaLaunchKernelEx(&cfg, kern, static_cast<KA>(args)...) != cudaSuccess) {
        cudaGetLastError();  // reported here; not left for the next call to find
        return DCNV4_ERR_LAUNCH;
    }
    return launch_status();
}

// Sizes of the predictor's projection: the checks every entry point that takes
// (M, C, G, K, flags, dtype) makes first, in the order of dcnv4_predictor.
int check_projection(int M, int C, int G, int K, unsigned flags, int dtype, long long* P, long long* NO) {
    if (M < 0 || C <= 0 || G <= 0 || K <= 0 || K > DCNV4_MAX_K) return DCNV4_ERR_SHAPE;
    if (flags & ~static_cast<unsigned>(DCNV4_FLAG_REMOVE_CENTER)) return DCNV4_ERR_FLAGS;
    const bool no_center = (flags & DCNV4_FLAG_REMOVE_CENTER) != 0u;
    if (no_center && (K % 2 == 0 || K < 3)) return DCNV4_ERR_SHAPE;
    if (!elem_size(dtype)) return DCNV4_ERR_DTYPE;
    *P = static_cast<long long>(K) * K - (no_center ? 1 : 0);
    *NO = 3LL * G * *P;
    if (static_cast<long long>(M) * C >= kLimit || *NO * C >= kLimit || static_cast<long long>(M) * *NO >= kLimit)
        return DCNV4_ERR_TOO_LARGE;
    return DCNV4_OK;
}
