// C entry points of the block norms (kernels: norms.cuh) and the column sums of their weights'
// gradients.
#include "norms.cuh"

namespace mfp8 {
namespace {

struct FinalArgs {
    const float* partial;      // [n][H]
    int n, H;
    const void *w, *gate;      // channel gate only
    int w_dtype, g_dtype;
    float w_offset, b;
    int channel, sigmoid;
    float *dw, *dgate;
};

// Column sums of the CTAs' partial sums: 32 columns per CTA, the rows dealt to 32 warps and
// joined in shared memory in warp order.
__global__ void __launch_bounds__(1024) norm_weight_grad_kernel(const FinalArgs a) {
    __shared__ float s[32][33];
    grid_dependency_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    float v = 0.0f;
    if (c < a.H) {
#pragma unroll 5
        for (int r = warp; r < a.n; r += 32) v += a.partial[static_cast<int64_t>(r) * a.H + c];
    }
    s[warp][lane] = v;
    __syncthreads();
    if (warp != 0 || c >= a.H) return;
    v = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i) v += s[i][lane];
    if (!a.channel) {
        a.dw[c] = v;
        return;
    }
    float g = weight_at(a.gate, a.g_dtype, c), slope = 1.0f;
    if (a.sigmoid) {
        const float e = exp_minus<float>(g);
        g = sigmoid_of<float>(e);
        slope = slope_of(e, g);
    }
    a.dw[c] = a.b * g * v;
    if (a.dgate) a.dgate[c] = slope * a.b * (weight_at(a.w, a.w_dtype, c) + a.w_offset) * v;
}

int check_norm(int T, int H, int dtype, int w_dtype) {
    if (T < 0 || H < 1 || !known_dtype(dtype) || !known_dtype(w_dtype)) return MOE_ERR_INVALID_ARG;
    if (H > MOE_MAX_HIDDEN_NORM) return MOE_ERR_UNSUPPORTED_SHAPE;
    return MOE_OK;
}

// Whether rows of these addresses (bits: addresses and byte strides, or-ed) go in 16-byte vectors.
bool wide_rows(uintptr_t bits, int H, size_t es) { return ((bits | (static_cast<uintptr_t>(H) * es)) & 15) == 0; }

cudaError_t launch_norm_dtype(const NormArgs& a, int dtype, int which, int gate, bool wide, cudaStream_t stream,
                              int* ctas) {
    const int sms = device_sms() < kPlanSms ? device_sms() : kPlanSms;   // the workspace holds kPlanSms partial rows
    if (dtype == MOE_DTYPE_FP32) return launch_norm_fp32(a, which, gate, wide, sms, stream, ctas);
    if (dtype == MOE_DTYPE_FP16) return launch_norm_fp16(a, which, gate, wide, sms, stream, ctas);
    return launch_norm_bf16(a, which, gate, wide, sms, stream, ctas);
}

cudaError_t launch_final(const FinalArgs& f, cudaStream_t stream) {
    return launch_pdl(norm_weight_grad_kernel, dim3(static_cast<unsigned>((f.H + 31) / 32)), dim3(1024), 0, stream, f);
}

// The gate's part of the arguments: MOE_OK, *gate = its shape (row for none).  A gate with a value per row or
// element holds none where there are no rows, and then needs no address.
int check_gate(const moe_post_norm_params* p, int T, int H, int* gate) {
    if (p->gate_kind < MOE_GATE_NONE || p->gate_kind > MOE_GATE_FULL) return MOE_ERR_INVALID_ARG;
    const bool by_row = p->gate_kind == MOE_GATE_TOKEN || p->gate_kind == MOE_GATE_FULL;
    if (p->gate_kind == MOE_GATE_NONE ? p->gate != nullptr : p->gate == nullptr && !(by_row && T == 0))
        return MOE_ERR_INVALID_ARG;
    if (p->gate_kind == MOE_GATE_TOKEN && p->gate_stride < 1) return MOE_ERR_INVALID_ARG;
    if (p->gate_kind == MOE_GATE_FULL && p->gate_stride < H) return MOE_ERR_INVALID_ARG;
    *gate = p->gate_kind == MOE_GATE_CHANNEL ? kGateChannel
            : p->gate_kind != MOE_GATE_FULL  ? kGateRow
            : p->gate_sigmoid                ? kGateFullSigmoid
                                             : kGateFull;
    return MOE_OK;
}
// Addresses and strides of the gate that decide on 16-byte vectors (a row gate is read by element).
uintptr_t gate_bits(const moe_post_norm_params* p, size_t es) {
    if (p->gate_kind == MOE_GATE_CHANNEL) return address(p->gate);
    if (p->gate_kind == MOE_GATE_FULL) return address(p->gate) | static_cast<uintptr_t>(p->gate_stride * es);
    return 0;
}

}  // namespace
}  // namespace mfp8

using namespace mfp8;

extern "C" {

int moe_pre_norm(const void* x, int64_t ldx, int dtype, const void* weight, int weight_dtype, float weight_offset,
                 float eps, int T, int H, void* h, float* rstd, void* stream) {
    int rc = check_norm(T, H, dtype, weight_dtype);
    if (rc != MOE_OK) return rc;
    if (ldx < H) return MOE_ERR_INVALID_ARG;
    if (T == 0) return MOE_OK;
    const size_t es = dtype_bytes(dtype);
    if (!x || !weight || !h || !rstd || !on_element(address(x) | address(h), es) ||
        !on_element(address(weight), dtype_bytes(weight_dtype)))
        return MOE_ERR_INVALID_ARG;
    uint32_t* status = nullptr;
    if ((rc = device_status_word(&status)) != MOE_OK) return rc;
    NormArgs a = {};
    a.status = status;
    a.T = T;
    a.H = H;
    a.x = x;
    a.ldx = ldx;
    a.w = weight;
    a.w_dtype = weight_dtype;
    a.w_offset = weight_offset;
    a.eps = eps;
    a.out = h;
    a.rstd = rstd;
    int ctas = 0;
    const bool wide = wide_rows(address(x) | address(h) | static_cast<uintptr_t>(ldx * es), H, es);
    return cuda_status(launch_norm_dtype(a, dtype, kPreForward, 0, wide, static_cast<cudaStream_t>(stream), &ctas));
}

size_t moe_norm_backward_workspace_size(int T, int H) {
    if (T < 1 || H < 1) return 0;
    return static_cast<size_t>(T < kPlanSms ? T : kPlanSms) * H * 4;
}

int moe_pre_norm_backward(const void* dh, int64_t lddh, const void* x, int64_t ldx, int dtype, const void* weight,
                          int weight_dtype, float weight_offset, const float* rstd, const void* dresidual,
                          int64_t lddres, int T, int H, void* dx, float* dweight, void* workspace,
                          size_t workspace_bytes, void* stream) {
    int rc = check_norm(T, H, dtype, weight_dtype);
    if (rc != MOE_OK) return rc;
    if (ldx < H || lddh < H || (dresidual && lddres < H) || !dweight) return MOE_ERR_INVALID_ARG;
    const size_t es = dtype_bytes(dtype);
    if (T > 0 && (!dh || !x || !weight || !rstd || !dx)) return MOE_ERR_INVALID_ARG;
    if (!on_element(address(dh) | address(x) | address(dresidual) | address(dx), es) ||
        !on_element(address(weight), dtype_bytes(weight_dtype)))
        return MOE_ERR_INVALID_ARG;
    if (workspace_bytes < moe_norm_backward_workspace_size(T, H)) return MOE_ERR_WORKSPACE_TOO_SMALL;
    if (T > 0 && !workspace) return MOE_ERR_INVALID_ARG;
    uint32_t* status = nullptr;
    if ((rc = device_status_word(&status)) != MOE_OK) return rc;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    int ctas = 0;
    if (T > 0) {
        NormArgs a = {};
        a.status = status;
        a.T = T;
        a.H = H;
        a.x = x;
        a.ldx = ldx;
        a.dout = dh;
        a.ldo = lddh;
        a.res = dresidual;
        a.ldr = lddres;
        a.w = weight;
        a.w_dtype = weight_dtype;
        a.w_offset = weight_offset;
        a.rstd = const_cast<float*>(rstd);
        a.out = dx;
        a.partial = static_cast<float*>(workspace);
        uintptr_t bits = address(dh) | address(x) | address(dx) | static_cast<uintptr_t>((ldx | lddh) * es);
        if (dresidual) bits |= address(dresidual) | static_cast<uintptr_t>(lddres * es);
        const cudaError_t e = launch_norm_dtype(a, dtype, kPreBackward, 0, wide_rows(bits, H, es), s, &ctas);
        if (e != cudaSuccess) return MOE_ERR_CUDA;
    }
    FinalArgs f = {};
    f.partial = static_cast<const float*>(workspace);
    f.n = ctas;
    f.H = H;
    f.dw = dweight;
    return cuda_status(launch_final(f, s));
}

int moe_post_norm(const void* y, int64_t ldy, const void* residual, int64_t ldr, int dtype,
                  const moe_post_norm_params* p, int T, int H, void* out, float* rstd, void* next_h, float* next_rstd,
                  void* stream) {
    if (!p) return MOE_ERR_INVALID_ARG;
    int gate = 0, rc = check_norm(T, H, dtype, p->weight_dtype);
    if (rc != MOE_OK || (rc = check_gate(p, T, H, &gate)) != MOE_OK) return rc;
    if (ldy < H || ldr < H) return MOE_ERR_INVALID_ARG;
    if (T == 0) return MOE_OK;
    const size_t es = dtype_bytes(dtype), ws = dtype_bytes(p->weight_dtype);
    if (!y || !residual || !p->weight || !out || !rstd || (p->next_weight && (!next_h || !next_rstd)))
        return MOE_ERR_INVALID_ARG;
    if (!on_element(address(y) | address(residual) | address(p->gate) | address(out) | address(next_h), es) ||
        !on_element(address(p->weight) | address(p->next_weight), ws))
        return MOE_ERR_INVALID_ARG;
    uint32_t* status = nullptr;
    if ((rc = device_status_word(&status)) != MOE_OK) return rc;
    NormArgs a = {};
    a.status = status;
    a.T = T;
    a.H = H;
    a.x = y;
    a.ldx = ldy;
    a.res = residual;
    a.ldr = ldr;
    a.gate = p->gate;
    a.ldg = p->gate_stride;
    a.w = p->weight;
    a.w2 = p->next_weight;
    a.w_dtype = p->weight_dtype;
    a.w_offset = p->weight_offset;
    a.eps = p->eps;
    a.a = p->residual_scale;
    a.b = p->block_scale;
    a.sigmoid = p->gate_sigmoid;
    a.out = out;
    a.h2 = next_h;
    a.rstd = rstd;
    a.rstd2 = next_rstd;
    uintptr_t bits = address(y) | address(residual) | address(out) | static_cast<uintptr_t>((ldy | ldr) * es) |
                     gate_bits(p, es);
    if (p->next_weight) bits |= address(next_h);
    int ctas = 0;
    return cuda_status(launch_norm_dtype(a, dtype, kPostForward, gate, wide_rows(bits, H, es),
                                         static_cast<cudaStream_t>(stream), &ctas));
}

int moe_post_norm_backward(const void* dout, int64_t lddout, const void* y, int64_t ldy, int dtype,
                           const moe_post_norm_params* p, const float* rstd, int T, int H, void* dy, void* dresidual,
                           void* dgate, float* dweight, void* workspace, size_t workspace_bytes, void* stream) {
    if (!p) return MOE_ERR_INVALID_ARG;
    int gate = 0, rc = check_norm(T, H, dtype, p->weight_dtype);
    if (rc != MOE_OK || (rc = check_gate(p, T, H, &gate)) != MOE_OK) return rc;
    if (lddout < H || ldy < H || !p->weight || !dweight || (dgate && p->gate_kind == MOE_GATE_NONE))
        return MOE_ERR_INVALID_ARG;
    const size_t es = dtype_bytes(dtype), ws = dtype_bytes(p->weight_dtype);
    if (T > 0 && (!dout || !y || !rstd || !dy)) return MOE_ERR_INVALID_ARG;
    const size_t gs = gate == kGateChannel ? 4 : es;   // a channel gate's gradient is fp32
    if (!on_element(address(dout) | address(y) | address(p->gate) | address(dy) | address(dresidual), es) ||
        !on_element(address(dgate), gs) || !on_element(address(p->weight), ws))
        return MOE_ERR_INVALID_ARG;
    if (workspace_bytes < moe_norm_backward_workspace_size(T, H)) return MOE_ERR_WORKSPACE_TOO_SMALL;
    if (T > 0 && !workspace) return MOE_ERR_INVALID_ARG;
    uint32_t* status = nullptr;
    if ((rc = device_status_word(&status)) != MOE_OK) return rc;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    int ctas = 0;
    if (T > 0) {
        NormArgs a = {};
        a.status = status;
        a.T = T;
        a.H = H;
        a.x = y;
        a.ldx = ldy;
        a.dout = dout;
        a.ldo = lddout;
        a.gate = p->gate;
        a.ldg = p->gate_stride;
        a.w = p->weight;
        a.w_dtype = p->weight_dtype;
        a.w_offset = p->weight_offset;
        a.a = p->residual_scale;
        a.b = p->block_scale;
        a.sigmoid = p->gate_sigmoid;
        a.out = dy;
        a.dres = dresidual;
        a.dgate = gate == kGateChannel ? nullptr : dgate;
        a.rstd = const_cast<float*>(rstd);
        a.partial = static_cast<float*>(workspace);
        uintptr_t bits = address(dout) | address(y) | address(dy) | static_cast<uintptr_t>((lddout | ldy) * es) |
                         address(dresidual) | gate_bits(p, es);
        if (full_gate(gate)) bits |= address(dgate);
        const cudaError_t e = launch_norm_dtype(a, dtype, kPostBackward, gate, wide_rows(bits, H, es), s, &ctas);
        if (e != cudaSuccess) return MOE_ERR_CUDA;
    }
    FinalArgs f = {};
    f.partial = static_cast<const float*>(workspace);
    f.n = ctas;
    f.H = H;
    f.w = p->weight;
    f.gate = p->gate;
    f.w_dtype = p->weight_dtype;
    f.g_dtype = dtype;
    f.w_offset = p->weight_offset;
    f.b = p->block_scale;
    f.channel = gate == kGateChannel;
    f.sigmoid = p->gate_sigmoid;
    f.dw = dweight;
    f.dgate = gate == kGateChannel ? static_cast<float*>(dgate) : nullptr;
    return cuda_status(launch_final(f, s));
}

}  // extern "C"
