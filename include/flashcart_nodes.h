/*
 * flashcart_nodes.h -- C ABI of libflashcart, part two: operators on node
 * rows that stand beside the edge convolution and the ladders of
 * flashcart.h.
 *   - fc_species_embed      node features from the species (element) table
 *   - fc_head_norm_rotate   RMS norm of query and key heads and their
 *                           rotation by the node positions, in one pass
 *   - fc_node_attention     all-pairs attention inside each structure of a
 *                           batch, with a bias by distance and capped scores
 * each with its vector-Jacobian product (_vjp).  Where the edge convolution
 * sums over the edges inside a cutoff, the attention sums over every node of
 * the receiver's structure.
 *
 * Conventions are those of flashcart.h (device pointers, streams, statuses,
 * caller-provided workspace, outputs overwritten) with these additions.
 * Types.  Rows (tables, heads, their gradients) are FP32, BF16 or FP16, one
 * type per call (FC_F32, FC_BF16, FC_F16).  Positions, weights (gamma),
 * slopes, log-sums and the gradients of all of these and of tables are FP32.
 * Sums, norms and softmax statistics are held in FP32 or FP64 whatever the
 * row type, and results are rounded once.  Inside the attention's matrix
 * products, weights and score gradients of 16-bit rows are 16-bit values (see
 * there), and FP32 operands are two TF32 terms (2^-20 of a value).
 * Heads.  A head is head_dim contiguous values, head_dim a multiple of 8 from
 * 8 to 128.  Head h of node n starts at n * ld + h * head_dim; the row step
 * ld (in values, a multiple of 8, at least heads * head_dim) lets queries,
 * keys and values be column blocks of one fused projection.  Offsets are
 * computed in 64 bits.
 * Memory.  Row arrays are 16-byte aligned, the others 4-byte aligned.
 * Outputs may not overlap inputs or each other.
 * Results.  No atomic additions of floating-point values: the same call gives
 * the same bits.  The attention kernels that wait on barriers give up after a
 * bounded time and set the word that fc_device_error reads.
 */
#ifndef FLASHCART_NODES_H
#define FLASHCART_NODES_H

#include "flashcart.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Types of row arrays. */
enum { FC_F32 = 0, FC_BF16 = 1, FC_F16 = 2 };

/* Node features from the species table:
 *   x[n, rank 0, k] = scale * table[species[n]][k],  every other rank 0,
 * x [n_nodes][(lmax+1)^2 C] in the node layout (the rank-0 block is the first
 * C values of a row), table [n_species][C], species [n_nodes] int32.
 * lmax 0..8 (0: a plain lookup); C a multiple of 4 (FP32) or 8 (16-bit
 * types).  A node whose species is outside [0, n_species) -- padding is
 * written as -1 -- gets a zero row. */
int fc_species_embed(int dtype, int n_nodes, int n_species, int lmax, int channels, float scale,
                     const int32_t *species, const void *table, void *x, fc_stream_t stream);

/* VJP of fc_species_embed:
 *   table_bar[s][k] = scale * sum_{n: species[n] = s} g[n, rank 0, k]
 * g like x (its other ranks are not read), table_bar [n_species][C] FP32
 * (species without nodes get 0; nodes of species outside the table add to
 * nothing).  The nodes are sorted by species (stable) and every row is summed
 * in that order.
 * workspace: fc_species_embed_vjp_workspace_size() bytes, 16-byte aligned,
 * ws_bytes = its real size (FC_ERR_WORKSPACE if NULL or smaller). */
size_t fc_species_embed_vjp_workspace_size(int n_nodes, int n_species, int channels);
int fc_species_embed_vjp(int dtype, int n_nodes, int n_species, int lmax, int channels, float scale,
                         const int32_t *species, const void *g, float *table_bar, void *workspace,
                         size_t ws_bytes, fc_stream_t stream);

/* Query and key heads of a row: heads 0 .. heads_q - 1 are queries, the
 * heads_k after them keys (either count may be 0, not both; at most 1024).  pairs: the
 * number R of rotated pairs, 0 <= 2 R <= head_dim. */
typedef struct {
  int dtype;
  int heads_q;
  int heads_k;
  int head_dim;
  int pairs;
  float eps; /* >= 0, added to the mean square */
} fc_head_desc;

/* RMS norm of every head and its rotation by the node's position:
 *   u_d = x_d gamma_d / sqrt(mean_d x_d^2 + eps)      (gamma of the head's kind)
 *   theta_f = sum_a pos[n][a] freq[a][f]              (f < R, a = x, y, z)
 *   y_f     = u_f cos(theta_f) - u_{f+R} sin(theta_f)
 *   y_{f+R} = u_f sin(theta_f) + u_{f+R} cos(theta_f),  y_d = u_d for d >= 2 R
 * so that the product of a rotated query and key depends on the difference of
 * their positions only.  That is invariance under translation, not under
 * rotation: with fixed frequency vectors the result depends on how a structure
 * is turned, unless the model averages over directions (the attention's bias by
 * distance has no such direction).  Angles are formed and reduced in FP64:
 * positions far from the origin lose nothing.  The mean square is formed in
 * FP32: |x| up to 1e18 (above, it overflows and the head comes out 0) and, if
 * eps is 0, from 1e-18 on.
 *   x [n_nodes] rows of (heads_q + heads_k) heads, step ldx; y likewise, step
 *   ldy; gamma_q, gamma_k [head_dim] (NULL: ones); pos [n_nodes][3] and freq
 *   [3][R] (needed if R > 0). */
int fc_head_norm_rotate(const fc_head_desc *desc, int n_nodes, const void *x, int64_t ldx,
                        const float *gamma_q, const float *gamma_k, const float *pos,
                        const float *freq, void *y, int64_t ldy, fc_stream_t stream);

/* VJP of fc_head_norm_rotate (frequencies are constants): given g, the
 * gradient of y (row step ldg), writes
 *   x_bar (row step ldxb), gamma_q_bar and gamma_k_bar [head_dim] (sums over
 *   all nodes and heads of the kind), pos_bar [n_nodes][3] (0 if R = 0);
 * each may be NULL to skip it.
 * workspace: fc_head_norm_rotate_vjp_workspace_size() bytes, 16-byte aligned. */
size_t fc_head_norm_rotate_vjp_workspace_size(const fc_head_desc *desc, int n_nodes);
int fc_head_norm_rotate_vjp(const fc_head_desc *desc, int n_nodes, const void *x, int64_t ldx,
                            const void *g, int64_t ldg, const float *gamma_q, const float *gamma_k,
                            const float *pos, const float *freq, void *x_bar, int64_t ldxb,
                            float *gamma_q_bar, float *gamma_k_bar, float *pos_bar,
                            void *workspace, size_t ws_bytes, fc_stream_t stream);

/* Attention descriptor.  heads (at most 1024) is a multiple of kv_heads:
 * receiver head h reads key and value head h / (heads / kv_heads). */
typedef struct {
  int dtype;
  int heads;
  int kv_heads;
  int head_dim;
  float scale; /* |scale| < 2e38 */
  float cap;   /* 0: scores as they are; > 0 (and < 2e38, scale / cap finite): cap tanh(score / cap) */
} fc_attn_desc;

/* Attention of the nodes of a batch of structures, receivers i to senders j
 * of the same structure:
 *   t_ij  = cap tanh(scale q_i.k_j / cap) - slope_h |p_i - p_j|
 *   out_i = sum_j exp(t_ij - lse_i) v_j,  lse_i = log sum_j exp(t_ij)
 * Structure b holds receivers recv_ptr[b] .. recv_ptr[b+1] - 1 and senders
 * send_ptr[b] .. send_ptr[b+1] - 1 (int32 [n_struct + 1] on the device,
 * non-decreasing; either side of a structure may be empty; n_struct at most
 * 2^31 - 65).  Receivers and
 * senders are counted apart, as in fc_edge_conv_rect: the same pointer twice
 * is self-attention, a few receivers against many senders is a probe, and a
 * receiver range of a graph cut over several GPUs attends to the gathered
 * senders.  Rows before the first structure and after the last belong to none
 * and are written as rows with nothing on the other side: out 0, lse
 * -infinity, gradients 0.  Pointers outside [0, n_recv] or [0, n_send] are
 * clamped: nothing faults, but the result is then meaningless.  A padded
 * batch gives each stretch of padding a structure of its own.
 *   q [n_recv] rows of heads, k and v [n_send] rows of kv_heads; steps ldq,
 *   ldk, ldv.  pos_recv [n_recv][3], pos_send [n_send][3], slope [heads]:
 *   the distance bias, all NULL for none; pos_send NULL: the senders are the
 *   receivers (n_send = n_recv) and pos_recv serves both.  Positions are
 *   finite, with distances below 1e18 (their squares are formed in FP32).
 *   send_mask [n_send] bytes, 0 hides a sender (its key and value rows are
 *   not used, whatever they hold); NULL hides none.
 *   out [n_recv] rows of heads, step ldo; lse [n_recv][heads] FP32 (natural
 *   log).  A receiver with no sender left gets a zero row and lse -infinity.
 *   out_f32 [n_recv][heads][head_dim] FP32, or NULL: the output before its
 *   rounding, which the VJP reads.  16-bit types then carry the weights
 *   through the value product as two 16-bit terms; without it as one (half a
 *   unit of 2^-8 or 2^-11 of each weight, averaged over the row), while their
 *   sum stays FP32.
 * workspace: fc_node_attention_workspace_size() bytes (0: none needed),
 * 16-byte aligned, ws_bytes = its real size. */
size_t fc_node_attention_workspace_size(const fc_attn_desc *desc, int n_struct, int n_recv, int n_send);
int fc_node_attention(const fc_attn_desc *desc, int n_struct, int n_recv, int n_send,
                      const int32_t *recv_ptr, const int32_t *send_ptr, const void *q, int64_t ldq,
                      const void *k, int64_t ldk, const void *v, int64_t ldv,
                      const float *pos_recv, const float *pos_send, const float *slope,
                      const uint8_t *send_mask, void *out, int64_t ldo, float *lse, float *out_f32,
                      void *workspace, size_t ws_bytes, fc_stream_t stream);

/* Host query: whether fc_node_attention (vjp 0) or its VJP (vjp not 0) runs on
 * the tcgen05 kernels, whose waits are bounded (fc_device_error): 1 or 0, and
 * -1 for a descriptor or sizes that the call refuses.  16-bit rows do from some
 * tens (wide heads) to hundreds (narrow heads) of rows of a structure on; a
 * call has one kernel, chosen by its average structure. */
int fc_node_attention_on_tcgen05(const fc_attn_desc *desc, int n_struct, int n_recv, int n_send, int vjp);

/* VJP of fc_node_attention.  With P_ij = exp(t_ij - lse_i), dt_ij =
 * P_ij (g_i.v_j - g_i.out_i) and ds_ij = scale (1 - tanh^2) dt_ij:
 *   q_bar_i = sum_j ds_ij k_j      k_bar_j = sum_{i, heads of the group} ds_ij q_i
 *   v_bar_j = sum_{i, heads of the group} P_ij g_i
 *   slope_bar_h    = -sum_ij dt_ij |p_i - p_j|
 *   pos_recv_bar_i = -sum_{j, h} slope_h dt_ij (p_i - p_j) / |p_i - p_j|
 *   pos_send_bar_j =  sum_{i, h} slope_h dt_ij (p_i - p_j) / |p_i - p_j|
 * (coincident nodes add nothing to the position gradients).  Without
 * pos_send, pos_recv_bar is the sum of both and pos_send_bar must be NULL.
 *   out_f32 and lse as fc_node_attention wrote them (FP32 rows: out_f32, or
 *   out itself if its rows are packed, ldo = heads * head_dim); g the gradient
 *   of out (step ldg); lse itself takes no gradient.
 *   q_bar, k_bar, v_bar packed ([n][heads][head_dim], rows' type), slope_bar
 *   [heads], pos_*_bar [n][3]: each may be NULL to skip it, which changes no
 *   bit of the others.  Hidden senders get 0.  16-bit types round P and ds / scale to the rows' type ahead of the
 *   products; FP16 then has 6e-8 as its smallest step and 65504 as its largest
 *   value, so that g should be scaled (as FP16 losses are) to keep P (g.v)
 *   between them.  Slopes and positions do not pass through 16 bits.
 * workspace: fc_node_attention_vjp_workspace_size() bytes, 16-byte aligned. */
size_t fc_node_attention_vjp_workspace_size(const fc_attn_desc *desc, int n_struct, int n_recv, int n_send);
int fc_node_attention_vjp(const fc_attn_desc *desc, int n_struct, int n_recv, int n_send,
                          const int32_t *recv_ptr, const int32_t *send_ptr, const void *q, int64_t ldq,
                          const void *k, int64_t ldk, const void *v, int64_t ldv,
                          const float *pos_recv, const float *pos_send, const float *slope,
                          const uint8_t *send_mask, const float *out_f32, const float *lse,
                          const void *g, int64_t ldg, void *q_bar, void *k_bar, void *v_bar,
                          float *pos_recv_bar, float *pos_send_bar, float *slope_bar,
                          void *workspace, size_t ws_bytes, fc_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* FLASHCART_NODES_H */
