// The last launch the stand-in launchers of the training and beam-search calls
// were asked for.
#ifndef STUB_TRAIN_RECORD_H
#define STUB_TRAIN_RECORD_H
#include <stdint.h>

struct stub_train_call {
  const char *what;
  int64_t n0, n1, n2, n3;
  int i0, i1;
  const void *p = nullptr;
};
extern stub_train_call g_train;

#endif
