// C ABI of the fused linear cross-entropy library (declared in include/flce.h):
// argument checks, the workspace plan, tensor-map encoding and the stream-ordered
// launch sequence.
//
// Launch sequence of flce_forward_backward (all on the caller's stream):
//   1. LSE GEMM   Z = H W^T, online max/sum-exp per (token block, vocabulary
//                 range) and the target logit      ("Liger Kernel: Fused Triton
//                 Kernels for LLM Training", The Architecture, 1.)
//   2. merge      per-token lse and NLL from the partials
//   3. reduce     n_valid, label check, loss, gradient scale (one block, fixed order)
//   4. for each token block b, for each vocabulary chunk c:
//        GRAD GEMM  recompute Z_bc, write G_bc = (softmax - onehot) * scale in bf16
//        dH + dW    one launch of both products (same page, 2.):
//                   dH_b  (+)= G_bc W_c     (fp32 accumulator over the chunks)
//                   dW_c  (+)= G_bc^T H_b   (fixed order over token blocks)
//      then, with several chunks, the rounding of the block's dH accumulator to bf16
// Nothing of size N x V is ever written: the largest buffer is one G chunk.
// flce_forward runs steps 1-3. On one vocabulary shard, flce_forward_shard runs
// step 1 with global label ids, a merge into the shard's (m, s, zt) and step 3
// for the label check; flce_backward_shard runs step 3 for the scale and step 4
// from the caller's combined lse, accumulating its dH part in fp32.
#include <algorithm>
#include <cstdint>
#include <cstring>

#include "flce_host.h"

namespace flce {

// Backward of a GEMM call, token block outer, vocabulary chunk inner: per chunk the
// gradient GEMM (G in bf16) and one launch of the dH and / or dW products.
int launch_backward_products(const Plan& P, const BackwardProducts& b, KernelTrace& trace) {
  const int64_t N = P.N, D = P.D, V = P.V;
  const uint16_t* H = b.H;
  const uint16_t* W = b.W;
  uint16_t* dH = b.dH;
  void* dW = b.dW;
  uint16_t* G = b.G;
  float* dh_acc = b.dh_acc;
  float* dw_acc = b.dw_acc;
  const bool to_f32 = b.dh_f32 != nullptr;   // fp32 dH part of a vocabulary shard
  const bool want_dh = dH != nullptr || to_f32;
  const bool dw_bf16 = b.dw_bf16;
  const int64_t tmo = b.timeout_ns;
  int32_t* status = b.status;
  const int sms = b.sms;
  cudaStream_t st = b.stream;
  const int cta = P.cta;
  const int pairs = std::max(1, sms / cta);
  const int64_t rows_b = ceil_div(P.n_block, P.tile_m) * P.tile_m;
  // MN-major operands: one 3-D copy per CTA when the MN extent is a multiple of
  // 64 (always for the G chunk), else 64-wide 2-D boxes.
  CUtensorMap mH_mn, mW_mn, mG_mn, mG_k, mG_out;
  const bool d_box3 = D % 64 == 0;
  const uint32_t b_chunks = static_cast<uint32_t>(BN / cta / 64);
  const bool ok_h = d_box3 ? encode_bf16_mn3(&mH_mn, H, D, N, D, BK, b_chunks)
                           : encode_bf16(&mH_mn, H, D, N, D, 64, BK);
  const bool ok_w = d_box3 ? encode_bf16_mn3(&mW_mn, W, D, V, D, BK, b_chunks)
                           : encode_bf16(&mW_mn, W, D, V, D, 64, BK);
  if (!ok_h || !ok_w || !encode_g_chunked(&mG_mn, G, rows_b, P.v_chunk, 64, BK, BM / 64, false) ||
      !encode_g_chunked(&mG_k, G, rows_b, P.v_chunk, 64, BM, 1, false) ||
      !encode_g_chunked(&mG_out, G, rows_b, P.v_chunk, 32, 32, 1, true))
    return FLCE_ERR_CUDA;
  // dW goes to fp32 dW, to bf16 dW (one token block), or to the fp32 accumulator
  // that bf16 dW is rounded from after the last token block.
  const bool dw_direct_bf16 = dw_bf16 && P.n_nblocks == 1;

  for (int blk = 0; blk < P.n_nblocks; ++blk) {
    const int64_t b0 = static_cast<int64_t>(blk) * P.n_block;
    const int nb_len = static_cast<int>(std::min<int64_t>(P.n_block, N - b0));
    for (int c = 0; c < P.n_chunks; ++c) {
      const int64_t c0 = static_cast<int64_t>(c) * P.v_chunk;
      const int c_len = static_cast<int>(std::min<int64_t>(P.v_chunk, V - c0));

      // G chunk: recompute Z_bc and form (softmax - onehot) * scale in bf16.
      GemmParams q = b.grad;
      q.a_mn_major = 0;
      q.b_mn_major = 0;
      q.a_mn0 = static_cast<int>(b0);
      q.b_mn0 = static_cast<int>(c0);
      q.m_blocks = static_cast<int>(ceil_div(nb_len, P.tile_m));
      q.n_blocks = static_cast<int>(ceil_div(c_len, BN));
      q.num_units = q.m_blocks * q.n_blocks;
      q.group_m = std::min(q.m_blocks, 16);
      q.timeout_ns = tmo;
      q.status = status;
      q.m_valid = nb_len;
      q.n_valid = c_len;
      q.row_base = static_cast<int>(b0);
      q.col_base = static_cast<int>(b.v_base + c0);
      q.out_row0 = 0;
      if (b.launch_grad(cta, *b.h_k, *b.w_k, mG_out, q, cta * std::min(q.num_units, pairs), st,
                        b.fp8) != cudaSuccess ||
          !trace())
        return FLCE_ERR_CUDA;

      const bool both = dW != nullptr && want_dh;
      GemmArgs aw{}, ah{};
      if (dW != nullptr) {
        // dW rows [c0, c0 + c_len) (+)= G_bc^T H_b: M = vocabulary, N = hidden, K = tokens.
        GemmParams& w = aw.p;
        w.a_mn_major = 1;
        w.b_mn_major = 1;
        w.a_box3 = 1;
        w.b_box3 = d_box3 ? 1 : 0;
        w.b_k0 = static_cast<int>(b0);
        w.m_blocks = static_cast<int>(ceil_div(c_len, P.tile_m));
        w.n_blocks = static_cast<int>(ceil_div(D, kWideDw ? 2 * BN : BN));
        w.k_blocks = static_cast<int>(ceil_div(nb_len, BK));
        w.num_units = w.m_blocks * w.n_blocks;
        w.group_m = std::min(w.m_blocks, 8);
        // every second tile of a pair walks K backwards, so a wave starts on the K
        // blocks the previous wave read last (still in L2); on the Llama-3-8B head
        // (N 8192, D 4096, 16128-id chunks) 19% fewer DRAM reads per launch
        w.k_serpentine = 1;
        w.idesc = make_idesc_bf16_f32(P.tile_m, BN, 1, 1);
        w.timeout_ns = tmo;
        w.status = status;
        w.m_valid = c_len;
        w.n_valid = static_cast<int>(D);
        // the map holds exactly the chunk's rows, so ragged tiles are clipped
        const int64_t dw_off = c0 * D;
        void* dw_base = dw_direct_bf16 ? static_cast<void*>(static_cast<uint16_t*>(dW) + dw_off)
                        : dw_bf16      ? static_cast<void*>(dw_acc + dw_off)
                                       : static_cast<void*>(static_cast<float*>(dW) + dw_off);
        if (!encode_out(&aw.c, dw_base, dw_direct_bf16, D, c_len, D)) return FLCE_ERR_CUDA;
        aw.a = mG_mn;
        aw.b = mH_mn;
        w.out_row0 = 0;
        w.out_mode = dw_direct_bf16 ? OUT_STORE_BF16 : (blk == 0 ? OUT_STORE_F32 : OUT_ADD_F32);
      }

      const bool wide_dh = both || kWideDhAlone;
      if (want_dh) {
        // dH rows [b0, b0 + nb_len) (+)= G_bc W_c: M = tokens, N = hidden, K = vocabulary.
        GemmParams& h = ah.p;
        h.a_mn_major = 0;
        h.a_kchunk = 1;
        h.b_mn_major = 1;
        h.b_box3 = d_box3 ? 1 : 0;
        h.b_k0 = static_cast<int>(c0);
        h.m_blocks = static_cast<int>(ceil_div(nb_len, P.tile_m));
        h.n_blocks = static_cast<int>(ceil_div(D, wide_dh ? 2 * BN : BN));
        h.k_blocks = static_cast<int>(ceil_div(c_len, BK));
        h.num_units = h.m_blocks * h.n_blocks;
        h.group_m = std::min(h.m_blocks, 8);
        h.k_serpentine = 1;   // as for dW (9% fewer DRAM reads on the same head)
        h.idesc = make_idesc_bf16_f32(P.tile_m, BN, 0, 1);
        h.timeout_ns = tmo;
        h.status = status;
        h.m_valid = nb_len;
        h.n_valid = static_cast<int>(D);
        // one chunk: bf16 dH directly; else an fp32 accumulator of this token
        // block's rows (stored by chunk 0, reduce-added by the others), rounded
        // to bf16 after the last chunk. The map holds exactly the block's rows.
        // A shard accumulates straight into its fp32 dH part.
        const bool dh_direct = P.n_chunks == 1 && !to_f32;
        const bool ok_dh = to_f32 ? encode_out(&ah.c, b.dh_f32 + b0 * D, false, D, nb_len, D)
                           : dh_direct ? encode_out(&ah.c, dH + b0 * D, true, D, nb_len, D)
                                       : encode_out(&ah.c, dh_acc, false, D, nb_len, D);
        if (!ok_dh) return FLCE_ERR_CUDA;
        ah.a = mG_k;
        ah.b = mW_mn;
        h.out_row0 = 0;
        h.out_mode = dh_direct ? OUT_STORE_BF16 : (c == 0 ? OUT_STORE_F32 : OUT_ADD_F32);
      }
      // dW and dH both read only G (and H, W), and write different outputs
      cudaError_t ge = cudaSuccess;
      if (both) {
        const int units = ah.p.num_units + aw.p.num_units;
        ge = launch_gemm_f32_pair(cta, ah, aw, cta * std::min(units, pairs), st);
      } else if (dW != nullptr) {
        ge = launch_gemm_f32(cta, aw.a, aw.b, aw.c, aw.p, cta * std::min(aw.p.num_units, pairs),
                             st, kWideDw ? 1 : 0);
      } else if (want_dh) {
        ge = launch_gemm_f32(cta, ah.a, ah.b, ah.c, ah.p, cta * std::min(ah.p.num_units, pairs),
                             st, wide_dh ? 1 : 0);
      }
      if (ge != cudaSuccess || ((dW != nullptr || want_dh) && !trace())) return FLCE_ERR_CUDA;
    }
    if (dH != nullptr && P.n_chunks > 1 &&
        (launch_f32_to_bf16(dh_acc, dH + b0 * D, static_cast<int64_t>(nb_len) * D, sms, st) !=
             cudaSuccess ||
         !trace()))
      return FLCE_ERR_CUDA;
  }
  if (dW != nullptr && dw_bf16 && !dw_direct_bf16 &&
      (launch_f32_to_bf16(dw_acc, static_cast<uint16_t*>(dW), V * D, sms, st) != cudaSuccess ||
       !trace()))
    return FLCE_ERR_CUDA;
  return FLCE_OK;
}

namespace {

// Fp8 carries the E4M3 operands of the FP8 variant (null for the bf16 path):
// they feed the two logits products; H and W (bf16) feed the gradient products.
struct Fp8Operands {
  const uint8_t* H8 = nullptr;
  const uint8_t* W8 = nullptr;
  const float* scale_h = nullptr;  // device fp32 scalars
  const float* scale_w = nullptr;
};

// A call on one vocabulary shard, rows [v_offset, v_offset + V) of a vocabulary of
// V_total ids (V_total == 0: an ordinary call over the whole vocabulary). The
// forward writes the shard's per-token (m, s, zt); the backward takes the combined
// lse and writes the shard's fp32 part of dH and its rows of dW.
struct Shard {
  int64_t v_offset = 0;
  int64_t V_total = 0;
  float* m = nullptr;
  float* s = nullptr;
  float* zt = nullptr;
  const float* lse_in = nullptr;
  float* dh_f32 = nullptr;
};

int run(const uint16_t* H, const uint16_t* W, const Fp8Operands& f8, const int32_t* labels,
        int64_t N, int64_t D, int64_t V, const flce_options* opt_in, float* loss, float* lse_out,
        uint16_t* dH, void* dW, bool backward, void* workspace, size_t ws_bytes, int32_t* status,
        void* stream_v, const Shard& sh = Shard{}) {
  flce_options o;
  flce_default_options(&o);
  if (opt_in != nullptr) o = *opt_in;
  const bool fp8 = f8.H8 != nullptr || f8.W8 != nullptr;
  if (!backward) {
    dH = nullptr;
    dW = nullptr;
  }
  const bool shard = sh.V_total > 0;
  // the backward of a shard writes fp32 dH parts instead of bf16 dH
  const bool want_dh = dH != nullptr || (shard && backward && sh.dh_f32 != nullptr);
  const bool need_bf16 = !fp8 || want_dh || dW != nullptr;
  if (labels == nullptr || (!shard && loss == nullptr) || workspace == nullptr)
    return FLCE_ERR_NULL;
  if (shard) {
    if (backward ? (sh.lse_in == nullptr || (!want_dh && dW == nullptr))
                 : (sh.m == nullptr || sh.s == nullptr || sh.zt == nullptr))
      return FLCE_ERR_NULL;
    if (sh.v_offset < 0 || sh.V_total > (int64_t(1) << 30) || sh.v_offset + V > sh.V_total)
      return FLCE_ERR_SHAPE;
    const uintptr_t a4 = reinterpret_cast<uintptr_t>(sh.m) | reinterpret_cast<uintptr_t>(sh.s) |
                         reinterpret_cast<uintptr_t>(sh.zt) | reinterpret_cast<uintptr_t>(sh.lse_in);
    if ((a4 & 3u) || (sh.dh_f32 && !aligned16(sh.dh_f32))) return FLCE_ERR_ALIGN;
  }
  // labels are ids of the whole vocabulary
  const int64_t V_lab = shard ? sh.V_total : V;
  const int64_t v_base = shard ? sh.v_offset : 0;   // id of W's row 0
  if (fp8 && (f8.H8 == nullptr || f8.W8 == nullptr)) return FLCE_ERR_NULL;
  if (need_bf16 && (H == nullptr || W == nullptr)) return FLCE_ERR_NULL;
  int rc = check_shape(N, D, V);
  if (rc != FLCE_OK) return rc;
  rc = check_options(o);
  if (rc != FLCE_OK) return rc;
  if (fp8 && (D % 16 != 0 || !aligned16(f8.H8) || !aligned16(f8.W8))) return FLCE_ERR_ALIGN;
  if (fp8 && (f8.scale_h == nullptr || f8.scale_w == nullptr)) return FLCE_ERR_NULL;
  if (fp8 && ((reinterpret_cast<uintptr_t>(f8.scale_h) & 3u) ||
              (reinterpret_cast<uintptr_t>(f8.scale_w) & 3u)))
    return FLCE_ERR_ALIGN;
  if ((H && !aligned16(H)) || (W && !aligned16(W)) || !aligned16(labels) ||
      !aligned16(workspace) ||
      (lse_out && !aligned16(lse_out)) || (dH && !aligned16(dH)) || (dW && !aligned16(dW)) ||
      (reinterpret_cast<uintptr_t>(loss) & 3u) || (reinterpret_cast<uintptr_t>(status) & 3u))
    return FLCE_ERR_ALIGN;
  int sms = 0;
  rc = device_info(&sms);
  if (rc != FLCE_OK) return rc;
  Plan P;
  rc = make_plan(N, D, V, o, sms, &P, backward);
  if (rc != FLCE_OK) return rc;
  if (ws_bytes < P.total) return FLCE_ERR_WORKSPACE;
  if (backward && o.reduction == FLCE_REDUCTION_NONE) {
    return FLCE_ERR_OPTION;  // a per-token loss needs a per-token upstream gradient
  }
  const bool per_token = o.reduction == FLCE_REDUCTION_NONE;

  cudaStream_t st = static_cast<cudaStream_t>(stream_v);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  float2* part = reinterpret_cast<float2*>(ws + P.off_part);
  float* zt = reinterpret_cast<float*>(ws + P.off_zt);
  // reduction "none": the merge writes each token's loss straight to the caller
  float* nll = per_token ? loss : reinterpret_cast<float*>(ws + P.off_nll);
  float* loss_scalar =
      (per_token || shard) ? reinterpret_cast<float*>(ws + P.off_scal + 8) : loss;
  float* lse = lse_out ? lse_out : reinterpret_cast<float*>(ws + P.off_lse);
  float* scal = reinterpret_cast<float*>(ws + P.off_scal);  // [0] scale
  int32_t* nvalid = reinterpret_cast<int32_t*>(ws + P.off_scal + 4);
  // per token (max, 1 / sum exp, 1 - p of the target) for the gradient epilogue;
  // a shard's backward has only the caller's combined lse
  float4* gstat = (backward && !shard) ? reinterpret_cast<float4*>(ws + P.off_gstat) : nullptr;
  uint16_t* G = reinterpret_cast<uint16_t*>(ws + P.off_g);
  float* dh_acc = reinterpret_cast<float*>(ws + P.off_dhacc);
  float* dw_acc = reinterpret_cast<float*>(ws + P.off_dwacc);
  const int64_t tmo = o.timeout_ns > 0 ? o.timeout_ns : kDefaultTimeoutNs;

  if (status != nullptr && cudaMemsetAsync(status, 0, sizeof(int32_t), st) != cudaSuccess)
    return FLCE_ERR_CUDA;
  // Optional per-kernel trace: event 0 before the first kernel, event k after kernel k.
  KernelTrace trace{o.trace_events, o.trace_capacity, st};
  if (!trace()) return FLCE_ERR_CUDA;

  const int cta = P.cta;
  const int pairs = std::max(1, sms / cta);
  // Operands of the two logits products: bf16 H, W, or E4M3 H8, W8 (128 bytes =
  // 128 elements per stage row).
  CUtensorMap mH_k, mW_k;
  if (fp8) {
    if (!encode_u8(&mH_k, f8.H8, D, N, D, 2 * BK, BM) ||
        !encode_u8(&mW_k, f8.W8, D, V, D, 2 * BK, static_cast<uint32_t>(BN / cta)))
      return FLCE_ERR_CUDA;
  } else if (!encode_bf16(&mH_k, H, D, N, D, BK, BM) ||
             !encode_bf16(&mW_k, W, D, V, D, BK, static_cast<uint32_t>(BN / cta))) {
    return FLCE_ERR_CUDA;
  }
  const int k_blocks_z = static_cast<int>(ceil_div(D, fp8 ? 2 * BK : BK));
  const uint32_t idesc_z = fp8 ? make_idesc_e4m3_f32(P.tile_m, BN) : make_idesc_bf16_f32(P.tile_m, BN, 0, 0);


  // ---- 1. forward LSE GEMM (the backward of a shard starts from the given lse) ----
  if (!(shard && backward)) {
    GemmParams g{};
    g.a_mn_major = 0;
    g.b_mn_major = 0;
    g.m_blocks = P.m_blocks;
    g.n_blocks = P.v_tiles;
    g.k_blocks = k_blocks_z;
    g.acc_scale_h = f8.scale_h;
    g.acc_scale_w = f8.scale_w;
    g.splits = P.splits;
    g.part_stride = P.part_stride;
    g.num_units = P.splits * P.m_blocks;
    g.group_m = std::min(P.m_blocks, 16);
    g.idesc = idesc_z;
    g.timeout_ns = tmo;
    g.status = status;
    g.m_valid = static_cast<int>(N);
    g.n_valid = static_cast<int>(V);
    g.labels = labels;
    g.row_base = 0;
    g.col_base = static_cast<int>(v_base);
    g.ignore_index = o.ignore_index;
    g.part = part;
    g.zt = zt;
    if (launch_gemm_lse(cta, mH_k, mW_k, g, cta * std::min(g.num_units, pairs), st, fp8 ? 1 : 0) !=
            cudaSuccess ||
        !trace())
      return FLCE_ERR_CUDA;

    // ---- 2. merge: lse and NLL, or a shard's (m, s, zt) ----
    const cudaError_t me =
        shard ? launch_shard_merge(part, zt, labels, static_cast<int>(N), static_cast<int>(v_base),
                                   static_cast<int>(v_base + V), P.part_stride, P.splits,
                                   o.ignore_index, sh.m, sh.s, sh.zt, st)
              : launch_lse_merge(part, zt, labels, static_cast<int>(N), static_cast<int>(V),
                                 P.part_stride, P.splits, o.ignore_index, lse, nll, gstat, st);
    if (me != cudaSuccess || !trace()) return FLCE_ERR_CUDA;
  }
  // ---- 3. reduce: label check, n, the gradient scale and (not for shards) the loss ----
  if (launch_loss_reduce(shard ? nullptr : nll, labels, static_cast<int>(N),
                         static_cast<int>(V_lab), o.ignore_index,
                         per_token ? FLCE_REDUCTION_SUM : o.reduction, o.grad_scale,
                         o.normalizer, loss_scalar, scal, nvalid, status,
                         st) != cudaSuccess ||
      !trace())
    return FLCE_ERR_CUDA;
  if (!want_dh && dW == nullptr) return FLCE_OK;
  BackwardProducts bp{};
  bp.H = H;
  bp.W = W;
  bp.h_k = &mH_k;
  bp.w_k = &mW_k;
  bp.launch_grad = launch_gemm_grad;
  bp.fp8 = fp8 ? 1 : 0;
  bp.grad.k_blocks = k_blocks_z;
  bp.grad.acc_scale_h = f8.scale_h;
  bp.grad.acc_scale_w = f8.scale_w;
  bp.grad.idesc = idesc_z;
  bp.grad.labels = labels;
  bp.grad.ignore_index = o.ignore_index;
  bp.grad.lse = shard ? sh.lse_in : lse;   // the lse the gradient is formed from
  bp.grad.gstat = gstat;
  bp.grad.scale = scal;
  bp.v_base = v_base;
  bp.dH = shard ? nullptr : dH;
  bp.dh_f32 = shard ? sh.dh_f32 : nullptr;
  bp.dW = dW;
  bp.dw_bf16 = o.dw_dtype == FLCE_DTYPE_BF16;
  bp.G = G;
  bp.dh_acc = dh_acc;
  bp.dw_acc = dw_acc;
  bp.timeout_ns = tmo;
  bp.status = status;
  bp.sms = sms;
  bp.stream = st;
  return launch_backward_products(P, bp, trace);
}

int workspace_bytes(int64_t N, int64_t D, int64_t V, const flce_options* opt, bool backward,
                    size_t* bytes) {
  if (bytes == nullptr) return FLCE_ERR_NULL;
  flce_options o;
  flce_default_options(&o);
  if (opt != nullptr) o = *opt;
  int rc = flce::check_shape(N, D, V);
  if (rc != FLCE_OK) return rc;
  rc = flce::check_options(o);
  if (rc != FLCE_OK) return rc;
  // The vocabulary-range split count depends on the SM count; plan for the
  // largest split count that choose_splits can return so that the size does not
  // depend on the device (and can be asked for without one).
  flce_options big = o;
  if (big.v_splits == 0) big.v_splits = static_cast<int32_t>(std::min<int64_t>(
                                            flce::ceil_div(V, flce::BN), 128));
  flce::Plan P;
  rc = flce::make_plan(N, D, V, big, 1, &P, backward);
  if (rc != FLCE_OK) return rc;
  *bytes = P.total;
  return FLCE_OK;
}

}  // namespace
}  // namespace flce

extern "C" {

void flce_default_options(flce_options* opt) {
  if (opt == nullptr) return;
  std::memset(opt, 0, sizeof(*opt));
  opt->ignore_index = -100;
  opt->reduction = FLCE_REDUCTION_MEAN;
  opt->grad_scale = 1.0f;
  opt->normalizer = 0.0f;
  opt->dw_dtype = FLCE_DTYPE_F32;
  opt->timeout_ns = 0;
}

int flce_workspace_size(int64_t N, int64_t D, int64_t V, const flce_options* opt, size_t* bytes) {
  return flce::workspace_bytes(N, D, V, opt, true, bytes);
}

int flce_forward_workspace_size(int64_t N, int64_t D, int64_t V, const flce_options* opt,
                                size_t* bytes) {
  return flce::workspace_bytes(N, D, V, opt, false, bytes);
}

int flce_get_plan(int64_t N, int64_t D, int64_t V, const flce_options* opt, int32_t want_dh,
                  int32_t want_dw, flce_plan_info* info) {
  if (info == nullptr) return FLCE_ERR_NULL;
  flce_options o;
  flce_default_options(&o);
  if (opt != nullptr) o = *opt;
  int rc = flce::check_shape(N, D, V);
  if (rc != FLCE_OK) return rc;
  rc = flce::check_options(o);
  if (rc != FLCE_OK) return rc;
  size_t ws = 0;
  rc = flce_workspace_size(N, D, V, &o, &ws);
  if (rc != FLCE_OK) return rc;
  int sms = 0;
  rc = flce::device_info(&sms);
  if (rc != FLCE_OK) return rc;
  flce::Plan P;
  rc = flce::make_plan(N, D, V, o, sms, &P, want_dh != 0 || want_dw != 0);
  if (rc != FLCE_OK) return rc;
  info->n_block = P.n_block;
  info->v_chunk = P.v_chunk;
  info->n_blocks = P.n_nblocks;
  info->n_chunks = P.n_chunks;
  info->v_splits = P.splits;
  // LSE GEMM, merge, reduce; per token block: per chunk the gradient GEMM and
  // one launch of the dW and / or dH products asked for, then (several chunks) the
  // bf16 rounding of dH; bf16 dW over several token blocks: one rounding of its
  // accumulator at the end.
  const int per_chunk = 1 + ((want_dh || want_dw) ? 1 : 0);
  const int per_block = P.n_chunks * per_chunk + ((want_dh && P.n_chunks > 1) ? 1 : 0);
  const bool dw_round = want_dw && o.dw_dtype == FLCE_DTYPE_BF16 && P.n_nblocks > 1;
  info->kernel_launches =
      3 + ((want_dh || want_dw) ? P.n_nblocks * per_block + (dw_round ? 1 : 0) : 0);
  info->workspace_bytes = ws;
  info->plan_bytes = P.total;
  return FLCE_OK;
}

int flce_ce_workspace_size(int64_t N, int64_t V, const flce_options* opt, size_t* bytes) {
  if (bytes == nullptr) return FLCE_ERR_NULL;
  flce_options o;
  flce_default_options(&o);
  if (opt != nullptr) o = *opt;
  if (N < 1 || V < 1 || N > (int64_t(1) << 30) || V > (int64_t(1) << 30)) return FLCE_ERR_SHAPE;
  const int rc = flce::check_options(o);
  if (rc != FLCE_OK) return rc;
  *bytes = 2 * flce::align_up(static_cast<size_t>(N) * 4, 256) + 256;
  return FLCE_OK;
}

int flce_ce_logits(const void* logits, int32_t dtype, int64_t ld, const int32_t* labels,
                   int64_t N, int64_t V, const flce_options* opt, float* loss, float* lse,
                   void* dlogits, int64_t dld, void* workspace, size_t ws_bytes, int32_t* status,
                   void* stream) {
  flce_options o;
  flce_default_options(&o);
  if (opt != nullptr) o = *opt;
  if (logits == nullptr || labels == nullptr || loss == nullptr || workspace == nullptr)
    return FLCE_ERR_NULL;
  if (N < 1 || V < 1 || N > (int64_t(1) << 30) || V > (int64_t(1) << 30)) return FLCE_ERR_SHAPE;
  int rc = flce::check_options(o);
  if (rc != FLCE_OK) return rc;
  if (dtype != FLCE_DTYPE_F32 && dtype != FLCE_DTYPE_BF16) return FLCE_ERR_OPTION;
  const int64_t elt = dtype == FLCE_DTYPE_BF16 ? 2 : 4;
  if (ld < V || (dlogits != nullptr && dld < V)) return FLCE_ERR_SHAPE;
  if ((ld * elt) % 16 != 0 || (dlogits != nullptr && (dld * elt) % 16 != 0)) return FLCE_ERR_ALIGN;
  if (!flce::aligned16(logits) || !flce::aligned16(labels) || !flce::aligned16(workspace) ||
      (dlogits && !flce::aligned16(dlogits)) || (lse && (reinterpret_cast<uintptr_t>(lse) & 3u)) ||
      (reinterpret_cast<uintptr_t>(loss) & 3u) || (reinterpret_cast<uintptr_t>(status) & 3u))
    return FLCE_ERR_ALIGN;
  if (dlogits == logits && dld != ld) return FLCE_ERR_OPTION;
  if (dlogits != nullptr && o.reduction == FLCE_REDUCTION_NONE) return FLCE_ERR_OPTION;
  size_t need = 0;
  rc = flce_ce_workspace_size(N, V, &o, &need);
  if (rc != FLCE_OK) return rc;
  if (ws_bytes < need) return FLCE_ERR_WORKSPACE;
  int sms = 0;
  rc = flce::device_info(&sms);
  if (rc != FLCE_OK) return rc;

  cudaStream_t st = static_cast<cudaStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const size_t nb = flce::align_up(static_cast<size_t>(N) * 4, 256);
  const bool per_token = o.reduction == FLCE_REDUCTION_NONE;
  float* nll = per_token ? loss : reinterpret_cast<float*>(ws);
  float* lse_ws = reinterpret_cast<float*>(ws + nb);
  float* scal = reinterpret_cast<float*>(ws + 2 * nb);
  int32_t* nvalid = reinterpret_cast<int32_t*>(ws + 2 * nb + 4);
  float* loss_scalar = per_token ? reinterpret_cast<float*>(ws + 2 * nb + 8) : loss;
  if (status != nullptr && cudaMemsetAsync(status, 0, sizeof(int32_t), st) != cudaSuccess)
    return FLCE_ERR_CUDA;
  flce::KernelTrace trace{o.trace_events, o.trace_capacity, st};
  if (!trace()) return FLCE_ERR_CUDA;
  const int Ni = static_cast<int>(N), Vi = static_cast<int>(V);
  if (dlogits != nullptr &&
      (flce::launch_ce_count(labels, Ni, Vi, o.ignore_index, o.reduction, o.grad_scale,
                             o.normalizer, scal, status, st) != cudaSuccess ||
       !trace()))
    return FLCE_ERR_CUDA;
  if (flce::launch_ce_rows(dtype == FLCE_DTYPE_BF16 ? 1 : 0, logits, ld * elt, labels, Ni, Vi,
                           o.ignore_index, scal, lse ? lse : lse_ws, nll, dlogits, dld * elt, sms,
                           status, o.timeout_ns > 0 ? o.timeout_ns : flce::kDefaultTimeoutNs,
                           st) != cudaSuccess ||
      !trace())
    return FLCE_ERR_CUDA;
  if (flce::launch_loss_reduce(nll, labels, Ni, Vi, o.ignore_index,
                               per_token ? FLCE_REDUCTION_SUM : o.reduction, o.grad_scale,
                               o.normalizer, loss_scalar, scal + 3, nvalid, status,
                               st) != cudaSuccess ||
      !trace())
    return FLCE_ERR_CUDA;
  return FLCE_OK;
}

int flce_forward_backward(const uint16_t* H, const uint16_t* W, const int32_t* labels, int64_t N,
                          int64_t D, int64_t V, const flce_options* opt, float* loss, float* lse,
                          uint16_t* dH, void* dW, void* workspace, size_t ws_bytes,
                          int32_t* status, void* stream) {
  return flce::run(H, W, flce::Fp8Operands{}, labels, N, D, V, opt, loss, lse, dH, dW, true,
                   workspace, ws_bytes, status, stream);
}

int flce_forward(const uint16_t* H, const uint16_t* W, const int32_t* labels, int64_t N, int64_t D,
                 int64_t V, const flce_options* opt, float* loss, float* lse, void* workspace,
                 size_t ws_bytes, int32_t* status, void* stream) {
  return flce::run(H, W, flce::Fp8Operands{}, labels, N, D, V, opt, loss, lse, nullptr, nullptr,
                   false, workspace, ws_bytes, status, stream);
}

int flce_forward_shard(const uint16_t* H, const uint16_t* W_shard, const int32_t* labels,
                       int64_t N, int64_t D, int64_t V_shard, int64_t v_offset, int64_t V_total,
                       const flce_options* opt, float* m, float* s, float* zt, void* workspace,
                       size_t ws_bytes, int32_t* status, void* stream) {
  if (V_total < 1) return FLCE_ERR_SHAPE;
  flce::Shard sh;
  sh.v_offset = v_offset;
  sh.V_total = V_total;
  sh.m = m;
  sh.s = s;
  sh.zt = zt;
  return flce::run(H, W_shard, flce::Fp8Operands{}, labels, N, D, V_shard, opt, nullptr, nullptr,
                   nullptr, nullptr, false, workspace, ws_bytes, status, stream, sh);
}

int flce_backward_shard(const uint16_t* H, const uint16_t* W_shard, const int32_t* labels,
                        int64_t N, int64_t D, int64_t V_shard, int64_t v_offset, int64_t V_total,
                        const flce_options* opt, const float* lse, float* dH_part, void* dW_shard,
                        void* workspace, size_t ws_bytes, int32_t* status, void* stream) {
  if (V_total < 1) return FLCE_ERR_SHAPE;
  flce::Shard sh;
  sh.v_offset = v_offset;
  sh.V_total = V_total;
  sh.lse_in = lse;
  sh.dh_f32 = dH_part;
  return flce::run(H, W_shard, flce::Fp8Operands{}, labels, N, D, V_shard, opt, nullptr, nullptr,
                   nullptr, dW_shard, true, workspace, ws_bytes, status, stream, sh);
}

int flce_forward_fp8(const uint8_t* H8, const float* scale_h, const uint8_t* W8,
                     const float* scale_w,
                     const int32_t* labels, int64_t N, int64_t D, int64_t V,
                     const flce_options* opt, float* loss, float* lse, void* workspace,
                     size_t ws_bytes, int32_t* status, void* stream) {
  flce::Fp8Operands f8;
  f8.H8 = H8;
  f8.W8 = W8;
  f8.scale_h = scale_h;
  f8.scale_w = scale_w;
  return flce::run(nullptr, nullptr, f8, labels, N, D, V, opt, loss, lse, nullptr, nullptr, false,
                   workspace, ws_bytes, status, stream);
}

int flce_forward_backward_fp8(const uint8_t* H8, const float* scale_h, const uint8_t* W8,
                              const float* scale_w,
                              const uint16_t* H, const uint16_t* W, const int32_t* labels,
                              int64_t N, int64_t D, int64_t V, const flce_options* opt,
                              float* loss, float* lse, uint16_t* dH, void* dW, void* workspace,
                              size_t ws_bytes, int32_t* status, void* stream) {
  flce::Fp8Operands f8;
  f8.H8 = H8;
  f8.W8 = W8;
  f8.scale_h = scale_h;
  f8.scale_w = scale_w;
  return flce::run(H, W, f8, labels, N, D, V, opt, loss, lse, dH, dW, true, workspace, ws_bytes,
                   status, stream);
}

int flce_quantize_e4m3(const uint16_t* x, int64_t n, uint8_t* q, float* out, void* stream) {
  if (x == nullptr || q == nullptr || out == nullptr) return FLCE_ERR_NULL;
  if (n < 1) return FLCE_ERR_SHAPE;
  if (n % 8 != 0 || !flce::aligned16(x) || !flce::aligned16(q) ||
      (reinterpret_cast<uintptr_t>(out) & 7u))
    return FLCE_ERR_ALIGN;
  int sms = 0;
  const int rc = flce::device_info(&sms);
  if (rc != FLCE_OK) return rc;
  return flce::launch_quantize_e4m3(x, n, q, out, sms, static_cast<cudaStream_t>(stream)) ==
                 cudaSuccess
             ? FLCE_OK
             : FLCE_ERR_CUDA;
}

int flce_scale_grads(uint16_t* dH, int64_t dh_elems, void* dW, int64_t dw_elems,
                     int32_t dw_dtype, const float* scale, void* stream) {
  if (scale == nullptr) return FLCE_ERR_NULL;
  if (dh_elems < 0 || dw_elems < 0) return FLCE_ERR_SHAPE;
  if ((dH == nullptr && dh_elems > 0) || (dW == nullptr && dw_elems > 0)) return FLCE_ERR_NULL;
  if (dw_dtype != FLCE_DTYPE_F32 && dw_dtype != FLCE_DTYPE_BF16) return FLCE_ERR_OPTION;
  const int64_t dw_bytes = dw_elems * (dw_dtype == FLCE_DTYPE_BF16 ? 2 : 4);
  if ((dh_elems * 2) % 16 != 0 || dw_bytes % 16 != 0) return FLCE_ERR_ALIGN;
  if ((dH && !flce::aligned16(dH)) || (dW && !flce::aligned16(dW)) ||
      (reinterpret_cast<uintptr_t>(scale) & 3u))
    return FLCE_ERR_ALIGN;
  int sms = 0;
  const int rc = flce::device_info(&sms);
  if (rc != FLCE_OK) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (dh_elems > 0 && flce::launch_scale(dH, dh_elems * 2, 1, scale, sms, st) != cudaSuccess)
    return FLCE_ERR_CUDA;
  if (dw_elems > 0 &&
      flce::launch_scale(dW, dw_bytes, dw_dtype == FLCE_DTYPE_BF16 ? 1 : 0, scale, sms, st) !=
          cudaSuccess)
    return FLCE_ERR_CUDA;
  return FLCE_OK;
}

int flce_check_status(const int32_t* status, void* stream) {
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (cudaStreamSynchronize(st) != cudaSuccess) return FLCE_ERR_CUDA;
  if (status == nullptr) return FLCE_OK;
  int32_t h = 0;
  if (cudaMemcpy(&h, status, sizeof(h), cudaMemcpyDeviceToHost) != cudaSuccess)
    return FLCE_ERR_CUDA;
  return h;
}

const char* flce_status_string(int code) {
  switch (code) {
    case FLCE_OK: return "ok";
    case FLCE_ERR_NULL: return "a required pointer is NULL";
    case FLCE_ERR_SHAPE: return "N, D or V out of range";
    case FLCE_ERR_ALIGN: return "pointer not 16-byte aligned or D not a multiple of 8";
    case FLCE_ERR_WORKSPACE: return "workspace too small";
    case FLCE_ERR_OPTION: return "option out of range";
    case FLCE_ERR_CUDA: return "CUDA call failed";
    case FLCE_ERR_DEVICE: return "device is not an sm_103 GPU";
    case FLCE_ERR_LABEL_RANGE: return "a label is outside [0, V) and is not ignore_index";
    case FLCE_ERR_TIMEOUT: return "a device pipeline wait timed out";
    default: return "unknown status";
  }
}

}  // extern "C"
