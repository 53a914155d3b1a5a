/*
 * Two host threads that call the layer operators at the same time, each with
 * memory and a stream of its own; their calls of one kernel need different
 * amounts of shared memory.  Every call has to be accepted.
 *
 *   layer_threads_client norm|gradients|experts CALLS
 * prints "N calls, M refused"; exit status 0 when none was.
 */
#include <cuda_runtime.h>
#include <pthread.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include "ar.h"

#define CUDA(call)                                                                   \
  do {                                                                               \
    cudaError_t e_ = (call);                                                         \
    if (e_ != cudaSuccess) {                                                         \
      fprintf(stderr, "CUDA error %s at %s:%d\n", cudaGetErrorString(e_), __FILE__, \
              __LINE__);                                                             \
      exit(2);                                                                       \
    }                                                                                \
  } while (0)

#define ROWS 500
#define HIDDEN 64
#define WIDTH 32
#define EXPERTS 8

struct work {
  const char* op;
  size_t size; /* columns of a norm, tokens of the experts */
  int calls, refused;
  pthread_barrier_t* begin;
};

static void* zeros(size_t bytes) {
  void* p;
  CUDA(cudaMalloc(&p, bytes));
  CUDA(cudaMemset(p, 0, bytes));
  return p;
}

static void* run(void* arg) {
  struct work* w = arg;
  cudaStream_t s;
  CUDA(cudaStreamCreate(&s));
  const size_t n = w->size;
  /* bfloat16 zeros: six matrices of ROWS x 8192 at most, and room for scratch */
  char* m[6];
  for (int i = 0; i < 6; ++i) m[i] = zeros((size_t)ROWS * 8192 * 2);
  const ar_norm_t norm = {AR_NORM_RMS, AR_BF16, ROWS, n, 0, 1e-5, 1.0, 0.0};
  const ar_norm_t few = {AR_NORM_RMS, AR_BF16, 4, n, 0, 1e-5, 1.0, 0.0};
  const ar_moe_t moe = {AR_BF16, AR_BF16, AR_ACT_SILU, EXPERTS, 0, EXPERTS, 2, 1, HIDDEN, WIDTH};
  const size_t room = (size_t)ROWS * 8192 * 2;
  CUDA(cudaDeviceSynchronize());
  pthread_barrier_wait(w->begin);
  for (int i = 0; i < w->calls; ++i) {
    ar_status_t st;
    if (!strcmp(w->op, "norm"))
      st = ar_residual_norm(&norm, m[0], n, m[1], n, NULL, 0, NULL, NULL, m[2], NULL, m[3], n, m[4], n, s);
    else if (!strcmp(w->op, "gradients"))
      st = ar_residual_norm_backward(&few, m[0], n, m[1], n, NULL, 0, m[2], n, NULL, 0, NULL, NULL, m[3], m[4], n, NULL, 0, NULL, 0,
                                     NULL, NULL, NULL, NULL, NULL, 0, s);
    else
      st = ar_moe_ffn(&moe, m[0], HIDDEN, m[1], EXPERTS, m[2], m[2], HIDDEN, HIDDEN * WIDTH, m[3], WIDTH, HIDDEN * WIDTH, m[4], HIDDEN,
                      NULL, NULL, n, m[5], room, s);
    w->refused += st != AR_OK;
    if (i % 256 == 255) CUDA(cudaStreamSynchronize(s));
  }
  CUDA(cudaStreamSynchronize(s));
  return NULL;
}

int main(int argc, char** argv) {
  if (argc != 3) return 3;
  const int experts = !strcmp(argv[1], "experts"), calls = atoi(argv[2]);
  pthread_barrier_t begin;
  pthread_barrier_init(&begin, NULL, 2);
  struct work w[2] = {{argv[1], experts ? 32 : 8192, calls, 0, &begin},
                      {argv[1], experts ? 1 : !strcmp(argv[1], "norm") ? 1024 : 6144, calls, 0, &begin}};
  pthread_t t[2];
  for (int i = 0; i < 2; ++i)
    if (pthread_create(&t[i], NULL, run, &w[i])) return 3;
  for (int i = 0; i < 2; ++i) pthread_join(t[i], NULL);
  CUDA(cudaDeviceSynchronize());
  printf("%d calls, %d refused\n", 2 * calls, w[0].refused + w[1].refused);
  return w[0].refused + w[1].refused ? 1 : 0;
}
